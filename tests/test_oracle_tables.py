"""The 64-bit references of the dense-table operators: hand-worked examples,
exact rational arithmetic, round trips."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import tables as ot


def test_round_to_bf16_worked():
    v = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -20, -3.0e38,
                  3.4e38, np.inf, np.nan], np.float32)
    want = [1.0, 1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, None, np.inf, np.inf, np.nan]
    got = ot.round_to(v, "bf16")
    for g, w in zip(got, want):
        if w is not None:
            assert (np.isnan(g) and np.isnan(w)) or g == w
    assert abs(got[4] + 3.0e38) <= 3.0e38 * 2.0 ** -8


def test_pack_worked():
    q = np.array([[1, 2, 3], [15, 0, 8]], np.uint8)
    assert ot.pack(q).tolist() == [[0x21, 0x03], [0x0F, 0x08]]
    assert np.array_equal(ot.unpack(ot.pack(q), 3), q)
    # the unused half byte of an odd row end is ignored
    assert np.array_equal(ot.unpack(np.array([[0x21, 0xF3], [0x0F, 0x98]], np.uint8), 3), q)


def test_values_and_product_against_fractions():
    rng = np.random.default_rng(3)
    rows, cols, group = 3, 70, 32
    codes = rng.integers(0, 256, (rows, 35)).astype(np.uint8)
    scales = rng.uniform(0.1, 1, (rows, 3)).astype(np.float32)
    zeros = rng.integers(0, 16, (rows, 3)).astype(np.uint8)
    x = rng.standard_normal(cols).astype(np.float32)
    a = ot.q4_values(codes, scales, zeros, group, cols)
    y, mag = ot.q4_run(a, x)
    for r in range(rows):
        total = Fraction(0)
        for k in range(cols):
            b = int(codes[r, k // 2])
            q = b >> 4 if k & 1 else b & 15
            v = Fraction(float(scales[r, k // group])) * (q - int(zeros[r, k // group]))
            assert float(v) == a[r, k]
            total += v * Fraction(float(x[k]))
        assert abs(float(total) - y[0, r]) <= 1e-13 * mag[0, r]


def test_quantize_worked():
    w = np.zeros((1, 32), np.float32)
    w[0, :4] = [7.0, -3.4, 2.5, 1.5]  # max 7: scale 1; 2.5 and 1.5 are ties and go to even
    codes, scales, zeros = ot.q4_quantize(w, 32, "f32", False)
    assert zeros is None and scales[0, 0] == 1.0
    assert ot.unpack(codes, 32)[0, :5].tolist() == [15, 5, 10, 10, 8]
    w[0, :4] = [10.0, -5.0, 0.5, 1.5]  # range 15: scale 1, zero 5
    codes, scales, zeros = ot.q4_quantize(w, 32, "f32", True)
    assert scales[0, 0] == 1.0 and zeros[0, 0] == 5
    assert ot.unpack(codes, 32)[0, :5].tolist() == [15, 0, 5, 7, 5]


@pytest.mark.parametrize("with_zeros", [False, True])
@pytest.mark.parametrize("scale_type", ["f32", "f16", "bf16"])
def test_quantize_error_within_half_a_step(with_zeros, scale_type):
    rng = np.random.default_rng(5)
    w = rng.standard_normal((6, 101)).astype(np.float32)
    codes, scales, zeros = ot.q4_quantize(w, 32, scale_type, with_zeros)
    back = ot.q4_values(codes, scales, zeros, 32, 101)
    step = scales[:, np.arange(101) // 32]
    # half a step, plus what rounding the scale (2^-8 of 15 steps) can push past the end codes
    slack = {"f32": 2.0 ** -20, "f16": 15 * 2.0 ** -11, "bf16": 15 * 2.0 ** -8}[scale_type]
    assert np.all(np.abs(back - w) <= step * (0.5 + slack + (0.5 if with_zeros else 0)))


def test_quantize_of_faulty_and_empty_groups():
    w = np.zeros((1, 96), np.float32)
    w[0, 40] = np.inf
    w[0, 70] = np.nan
    for z in (False, True):
        codes, scales, zeros = ot.q4_quantize(w, 32, "f32", z)
        back = ot.q4_values(codes, scales, zeros, 32, 96)
        assert np.all(back[0, :32] == 0) and np.all(np.isnan(back[0, 32:]))


def test_embed_and_gradient_are_the_one_hot_products():
    rng = np.random.default_rng(9)
    vocab, dim = 7, 5
    tokens = np.array([3, -1, 0, 3, 6, 7, 3, 2 ** 40])
    table = rng.standard_normal((vocab, dim)).astype(np.float32)
    hot = np.zeros((len(tokens), vocab))
    for t, v in enumerate(tokens):
        if 0 <= v < vocab:
            hot[t, v] = 2.0
    assert np.allclose(ot.embed(table, tokens, 2.0, "f32"), hot @ table, rtol=0, atol=1e-6)
    g = rng.standard_normal((len(tokens), dim))
    grad, mag, count = ot.embed_grad(g, tokens, vocab, 2.0)
    assert np.allclose(grad, hot.T @ g, rtol=0, atol=1e-14)
    assert count.tolist() == [1, 0, 0, 3, 0, 0, 1]
    base = rng.standard_normal((vocab, dim))
    added, _, _ = ot.embed_grad(g, tokens, vocab, 2.0, base)
    assert np.allclose(added, grad + base, rtol=0, atol=1e-14)


@pytest.mark.parametrize("with_zeros,steps", [(False, 7), (True, 15)])
def test_quantize_scale_against_fractions(with_zeros, steps):
    """The factor is the fp32 number nearest to 1/7 or 1/15 and the scale is the range
    times it, rounded once to fp32 and once to its type: within a unit of fp32 of the
    range's exact quotient, as a division by a constant in fp32 is computed on a GPU."""
    factor = Fraction(float(np.float32(1 / steps)))
    near = [Fraction(float(np.nextafter(np.float32(1 / steps), np.float32(d)))) for d in (0, 1)]
    assert all(abs(factor - Fraction(1, steps)) < abs(v - Fraction(1, steps)) for v in near)
    rng = np.random.default_rng(12)
    w = (rng.standard_normal((300, 32)) * 10.0 ** rng.integers(-20, 20, (300, 1))).astype(
        np.float32)
    for scale_type in ("f32", "bf16"):
        _, scales, _ = ot.q4_quantize(w, 32, scale_type, with_zeros)
        for row, got in zip(w, scales[:, 0]):
            low, high = min(row.min(), 0.0), max(row.max(), 0.0)
            width = (Fraction(float(np.float32(high - low))) if with_zeros
                     else Fraction(float(max(high, -low))))
            raw = np.float32(float(width * factor))  # (48 bits: exact in float64)
            assert got == ot.round_to(np.array([raw]), scale_type)[0]
            assert abs(Fraction(float(raw)) - width / steps) <= Fraction(2) ** -23 * width / steps
