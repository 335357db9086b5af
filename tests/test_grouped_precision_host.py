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


@pytest.mark.parametrize("n,k,g", GC.SHAPES)
def test_wide_x_tells_a_missing_part(n, k, g):
    off, t, x, s, w = case(GC.wide_x, "some", n, k, g)
    hi, mid, lo = GC.parts(x)
    used = x != 0
    assert lo[used].all() and mid[used].all()
    want = GC.exact(x, w, off, t, n)
    assert np.abs(want).max() < 2.0 ** 23 and np.array_equal(2 * want, np.rint(2 * want))
    own = (GC.exact(np.ones_like(x), np.ones_like(w), off, t, n) > 0) & (want != 0)
    for model in (hi, hi + mid, hi + lo, GC.bf16(x)):
        assert (GC.exact(model, w, off, t, n) != want)[own].mean() > 0.9


@pytest.mark.parametrize("k,g", [(4096, 128), (2048, 64), (1120, 32), (1280, 256)])
def test_real_bound_tells_bf16_x(k, g):
    """On normal data the bound that grows with the root of K passes float32 arithmetic and refuses x or weights of bf16,
    and zeros."""
    off, t, n = np.array([0, 16], np.int32), 16, 60
    rng = np.random.default_rng(k)
    x, wf = GC.real_float_x(rng, t, 1, n, k)
    b = wf.reshape(n, -1, g)
    s = ((b.max(-1) - b.min(-1)) / 15).astype(np.float16).astype(np.float32)
    z = np.clip(np.rint(-b.min(-1) / s), 0, 15).astype(np.float32)
    code = np.clip(np.rint(b / s[..., None] + z[..., None]), 0, 15).astype(np.uint8).reshape(1, n, k)
    w = GC.weights(code, s[None], z[None], g)
    want, allowed = GC.exact(x, w, off, t, n), GC.allowance_real(x, s[None], g, off)
    for model_x, model_w in ((GC.bf16(x), w), (GC.parts(x)[0], w), (x, rounded(w)), (0 * x, w)):
        assert (np.abs(GC.exact(model_x, model_w, off, t, n) - want) > allowed).mean() > 0.8
    xb, cb = x.reshape(t, -1, g), code.reshape(n, -1, g).astype(np.float32)
    for bias in (np.float32(0), np.float32(16)):  # group by group in float32
        y = np.zeros((t, n), np.float32)
        for j in range(k // g):
            d = np.zeros((t, n), np.float32)
            xs = np.zeros(t, np.float32)
            for i in range(0, g, 32):
                d += (xb[:, j, i:i + 32].astype(np.float64) @ (bias + cb[:, j, i:i + 32]).T.astype(np.float64)).astype(np.float32)
                xs += xb[:, j, i:i + 32].astype(np.float64).sum(1).astype(np.float32)
            y += s[:, j] * d - s[:, j] * (bias + z[:, j]) * xs[:, None]
        assert (np.abs(y - want) <= allowed).all()
