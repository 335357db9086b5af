"""CPU checks of grouped_cases: models of the INT4 product that round a weight
fail the criteria which the GPU tests apply, and exact ones pass."""
import numpy as np
import pytest

import oracle.mxfp4_oracle as MX
import tests.grouped_cases as GC


def rounded(w):
    return GC.bf16(w.astype(np.float32)).astype(np.float64)


def in_two(w):
    """The weight as the sum of two bf16 values."""
    hi = rounded(w)
    return hi + rounded(w - hi)


def case(make, split, n, k, g):
    off, t = GC.offsets_of(split)
    x, code, s, z = make(np.random.default_rng(n + k + g + t), t, len(off) - 1, n, k, g)
    return off, t, x, s, GC.weights(code, s, z, g)


@pytest.mark.parametrize("n,k,g", GC.SHAPES)
def test_half_scales_tell_rounded_weights(n, k, g):
    off, t, x, s, w = case(GC.sparse_scales_f16, "some", n, k, g)
    want = GC.exact(x, w, off, t, n)
    assert np.array_equal(np.ldexp(want, 13), np.rint(np.ldexp(want, 13))) and np.abs(want).max() < 2.0 ** 7
    got = GC.exact(x, rounded(w), off, t, n)
    assert (GC.bf16(got) != GC.bf16(want)).mean() > 0.05
    assert np.array_equal(GC.exact(x, in_two(w), off, t, n), want)  # two parts hold 11 + 4 bits


@pytest.mark.parametrize("n,k,g", GC.SHAPES)
def test_float_scales_tell_weights_in_two_parts(n, k, g):
    off, t, x, s, w = case(GC.sparse_scales_f32, "some", n, k, g)
    want, allowed = GC.exact(x, w, off, t, n), GC.allowance_f32(x, s, g, off)
    own = allowed > 0
    for model in (rounded, in_two):
        assert (np.abs(GC.exact(x, model(w), off, t, n) - want) > allowed)[own].mean() > 0.3


@pytest.mark.parametrize("n,k,g", GC.SHAPES)
def test_float_scales_pass_in_float32(n, k, g):
    """The two float32 forms of the product, with their roundings: sums of codes times the scale less the zero-point's
    part, and sums of 16 + code with 16 + zero-point."""
    off, t = GC.offsets_of("some")
    e = len(off) - 1
    x, code, s, z = GC.sparse_scales_f32(np.random.default_rng(n + k + g + t), t, e, n, k, g)
    want, allowed = GC.exact(x, GC.weights(code, s, z, g), off, t, n), GC.allowance_f32(x, s, g, off)
    expert = np.searchsorted(off, np.arange(t), side="right") - 1
    for row in np.flatnonzero((expert >= 0) & (expert < e)):
        col = int(np.flatnonzero(x[row])[0])
        xv, q = x[row, col], code[expert[row], :, col].astype(np.float32)
        sv, zv = s[expert[row], :, col // g], z[expert[row], :, col // g]
        for bias in (np.float32(0), np.float32(16)):
            y = sv * (xv * (bias + q)) - sv * (bias + zv) * xv  # every operation rounds to float32
            assert y.dtype == np.float32 and (np.abs(y - want[row]) <= allowed[row]).all()


def test_bf16_rounds_to_the_nearest():
    a = np.array([1.0, 1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, 1.0 + 2.0 ** -9, -1.0 - 2.0 ** -8 - 2.0 ** -20], np.float32)
    assert GC.bf16(a).tolist() == [1.0, 1.0, 1.0 + 2.0 ** -6, 1.0, -1.0 - 2.0 ** -7]
