"""4-bit matrices: conversion (bit for bit), products with vectors and rows
back in dense form, against the 64-bit references.

Bound of a product, per entry: a group's terms are exact and summed in fp32
(at most group/16 = 8 steps of 16 terms, 2 * 2^-23 of the magnitudes each),
the groups' sums are scaled and added (one step each) and at most 32 partial
sums are joined: (8 + groups + 32) * 2^-22 * sum |A x| + |c|, then half a unit
of the result's type."""
import numpy as np
import pytest
import torch

from oracle import tables as ot

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sp():
    from conftest import build_library
    build_library()
    import spmv_sparse_storage_gb300 as sp
    torch.cuda.set_device(0)
    return sp


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(TYPES[dtype])


def host(t):
    return t.float().cpu().numpy()


def padded(rows, cols, dtype, ld, fill):
    """A [rows, cols] view of rows that are ld long, everything set to fill."""
    return torch.full((rows, ld), fill, dtype=dtype, device="cuda")[:, :cols]


def make(seed, rows, cols, group, scale_type, zeros):
    rng = np.random.default_rng(seed)
    groups = -(-cols // group)
    codes = rng.integers(0, 256, (rows, (cols + 1) // 2)).astype(np.uint8)
    scales = ot.round_to(rng.uniform(0.002, 0.02, (rows, groups)) *
                         rng.choice([-1, 1], (rows, groups)), scale_type)
    z = rng.integers(0, 16, (rows, groups)).astype(np.uint8) if zeros else None
    return codes, scales, z


def check_product(got, values, x, c, groups, y_type):
    want, mag = ot.q4_run(values, x, c)
    bound = (8 + groups + 32) * 2.0 ** -22 * mag
    bound = bound + ot.half_ulp(np.abs(want) + bound, y_type)
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(err <= bound), float((err / bound).max())


SHAPES = [(1, 1), (1, 2), (3, 31), (16, 32), (17, 33), (5, 64), (33, 100), (64, 127), (130, 128),
          (16, 129), (200, 255), (7, 1000), (100, 1024), (2, 4099), (513, 2080), (40, 8192),
          (9, 16500)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("group,scale_type,zeros,x_type,y_type", [
    (32, "bf16", False, "bf16", "bf16"), (64, "f16", True, "f16", "f16"),
    (128, "f32", False, "f32", "f32"), (128, "f16", True, "bf16", "f32"),
    (32, "f32", True, "f32", "bf16"), (64, "bf16", False, "f16", "f32")])
def test_products(sp, rows, cols, group, scale_type, zeros, x_type, y_type):
    codes, scales, z = make(rows * 131 + cols, rows, cols, group, scale_type, zeros)
    values = ot.q4_values(codes, scales, z, group, cols)
    rng = np.random.default_rng(cols)
    dc, ds, dz = dev(codes), dev(scales, scale_type), None if z is None else dev(z)
    for n, residual in [(1, False), (1, True), (2, False), (3, True), (8, False), (9, True),
                        (16, False), (19, True)]:
        if n > 3 and rows * cols > 300_000:
            continue
        x = ot.round_to(rng.standard_normal((n, cols)), x_type)
        c = ot.round_to(rng.standard_normal((n, rows)), y_type) if residual else None
        y = torch.full((n, rows), float("nan"), dtype=TYPES[y_type], device="cuda")
        sp.spmv_q4_run(dc, ds, group, dev(x, x_type), y,
                       c=None if c is None else dev(c, y_type), zeros=dz)
        check_product(host(y), values, x, c, scales.shape[1], y_type)


@pytest.mark.parametrize("pad", [0, 1, 3, 8, 16])
@pytest.mark.parametrize("shift", [0, 1, 4, 8])
def test_strides_and_offsets(sp, pad, shift):
    """Rows further apart than they are long, arrays that do not start on a
    vector's boundary, garbage (NaN) in every gap: neither read into a result
    nor written."""
    rows, cols, group, n = 37, 333, 64, 3
    codes, scales, z = make(7, rows, cols, group, "f16", True)
    values = ot.q4_values(codes, scales, z, group, cols)
    x = ot.round_to(np.random.default_rng(1).standard_normal((n, cols)), "bf16")
    c = ot.round_to(np.random.default_rng(2).standard_normal((n, rows)), "bf16")

    def place(a, dtype, fill):
        r, w = a.shape
        flat = torch.full((shift + r * (w + pad),), fill, dtype=dtype, device="cuda")
        view = flat[shift:].view(r, w + pad)[:, :w]
        view.copy_(dev(a).to(dtype))
        return flat, view

    _, dc = place(codes, torch.uint8, 0xFF)
    _, ds = place(scales, torch.float16, float("nan"))
    _, dz = place(z, torch.uint8, 0xFF)
    _, dx = place(x, torch.bfloat16, float("nan"))
    _, dcc = place(c, torch.bfloat16, float("nan"))
    flat, y = place(np.zeros((n, rows), np.float32), torch.bfloat16, 123.0)
    sp.spmv_q4_run(dc, ds, group, dx, y, c=dcc, zeros=dz)
    check_product(host(y), values, x, c, scales.shape[1], "bf16")
    gaps = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    gaps[shift:].view(n, rows + pad)[:, :rows] = False
    assert torch.all(flat[gaps] == 123.0)
    # accumulate in place
    sp.spmv_q4_run(dc, ds, group, dx, dcc, c=dcc, zeros=dz)
    assert torch.equal(dcc, y)


def test_accumulation_is_y_plus_ax(sp):
    """c = y is the library's multiply-and-accumulate, also for many vectors."""
    codes, scales, z = make(8, 50, 256, 128, "f32", False)
    values = ot.q4_values(codes, scales, z, 128, 256)
    rng = np.random.default_rng(4)
    x = rng.standard_normal((21, 256)).astype(np.float32)
    y0 = rng.standard_normal((21, 50)).astype(np.float32)
    y = dev(y0)
    sp.spmv_q4_run(dev(codes), dev(scales), 128, dev(x), y, c=y)
    check_product(host(y), values, x, y0, 2, "f32")


@pytest.mark.parametrize("rows,cols", [(1, 40), (70, 333), (33, 1024), (300, 96)])
@pytest.mark.parametrize("x_type,y_type,per_pass", [("bf16", "f32", 16), ("f16", "f16", 16),
                                                    ("f32", "f32", 5)])
def test_many_vectors(sp, rows, cols, x_type, y_type, per_pass):
    """A prompt's worth of vectors, at the numbers where another reading of the matrix
    begins, in rows further apart than they are long: each the product that it is alone
    or with the others of its reading, bit for bit, and nothing written between them."""
    codes, scales, z = make(31, rows, cols, 32, "f16", True)
    values = ot.q4_values(codes, scales, z, 32, cols)
    dc, ds, dz = dev(codes), dev(scales, "f16"), dev(z)
    rng = np.random.default_rng(rows)
    for n in (per_pass, per_pass + 1, 4 * per_pass, 4 * per_pass + 1, 100, 257):
        x = ot.round_to(rng.standard_normal((n, cols)), x_type)
        c = ot.round_to(rng.standard_normal((n, rows)), y_type)
        dx = padded(n, cols, TYPES[x_type], cols + 3, float("nan"))
        dx.copy_(dev(x))
        y = padded(n, rows, TYPES[y_type], rows + 5, 99.0)
        sp.spmv_q4_run(dc, ds, 32, dx, y, c=dev(c, y_type), zeros=dz)
        check_product(host(y), values, x, c, scales.shape[1], y_type)
        assert torch.all(y._base[:, rows:] == 99.0)
        first = n - 1 - (n - 1) % per_pass  # of the last reading
        part = torch.empty(n - first, rows, dtype=TYPES[y_type], device="cuda")
        sp.spmv_q4_run(dc, ds, 32, dx[first:], part, c=dev(c[first:], y_type), zeros=dz)
        assert torch.equal(part, y[first:])


@pytest.mark.parametrize("x_type", ["f32", "f16", "bf16"])
def test_infinities_and_nan(sp, x_type):
    """An infinity or a NaN in x or in a scale reaches exactly the results
    whose formula has it."""
    rows, cols, group = 40, 200, 32
    codes, scales, _ = make(9, rows, cols, group, "f32", False)
    codes[:, 10] |= 0x01  # column 20: code 1 or more below 8, never 8
    codes[:, 10] &= 0xF1
    x = ot.round_to(np.random.default_rng(3).standard_normal((3, cols)), x_type)
    x[1, 20] = np.inf
    x[2, 20] = np.nan
    scales[5, 2] = np.nan
    values = ot.q4_values(codes, scales, None, group, cols)
    y = torch.zeros(3, rows, device="cuda")
    sp.spmv_q4_run(dev(codes), dev(scales), group, dev(x, x_type), y)
    got = host(y)
    clean = np.arange(rows) != 5
    want, _ = ot.q4_run(values, x[:1])
    assert np.all(np.isfinite(got[0, clean])) and np.isnan(got[0, 5])
    assert np.allclose(got[0, clean], want[0, clean], rtol=1e-4, atol=1e-4)
    signs = np.sign(values[:, 20])
    assert np.all(signs[clean] != 0)
    assert np.array_equal(got[1, clean], signs[clean] * np.inf)
    assert np.all(np.isnan(got[2]))


def test_fp32_vectors_keep_their_low_bits(sp):
    """x = 1 + 2^-23 * k and codes that cancel the leading bit: only a product
    of all 24 bits of x gives the difference."""
    rows, cols = 16, 64
    codes = np.full((rows, cols // 2), 0x88, np.uint8)
    codes[:, 0] = 0x79  # +1 at column 0, -1 at column 1
    scales = np.ones((rows, 1), np.float32)
    x = np.ones((1, cols), np.float32)
    x[0, 0] = 1 + 5 * 2.0 ** -23
    y = torch.zeros(1, rows, device="cuda")
    sp.spmv_q4_run(dev(codes), dev(scales), 64, dev(x), y)
    assert np.all(host(y) == 5 * 2.0 ** -23)


@pytest.mark.parametrize("scale", [1e-38, 1e-20, 1e30])
def test_fp32_vectors_of_any_size(sp, scale):
    rows, cols = 20, 96
    codes, scales, _ = make(10, rows, cols, 32, "f32", False)
    values = ot.q4_values(codes, scales, None, 32, cols)
    x = (np.random.default_rng(6).standard_normal((2, cols)) * scale).astype(np.float32)
    y = torch.zeros(2, rows, device="cuda")
    sp.spmv_q4_run(dev(codes), dev(scales), 32, dev(x), y)
    want, mag = ot.q4_run(values, x)
    # subnormal terms may be flushed: 2^-126 for each of the columns' 8 steps and halves
    bound = (8 + 3 + 32) * 2.0 ** -22 * mag + cols * 16 * 2.0 ** -126
    assert np.all(np.abs(host(y) - want) <= bound)


def test_nothing_to_do(sp):
    codes, scales, _ = make(11, 5, 40, 32, "f32", False)
    dc, ds = dev(codes), dev(scales)
    y = torch.full((0, 5), 1.0, device="cuda")
    sp.spmv_q4_run(dc, ds, 32, torch.zeros(0, 40, device="cuda"), y)
    # no columns: y = c, or zeros
    c = torch.arange(5.0, device="cuda").view(1, 5)
    y = torch.full((1, 5), 7.0, device="cuda")
    empty = torch.empty(5, 0, dtype=torch.uint8, device="cuda")
    sp.spmv_q4_run(empty, torch.empty(5, 0, device="cuda"), 32, torch.empty(1, 0, device="cuda"),
                   y, c=c)
    assert torch.equal(y, c)
    sp.spmv_q4_run(empty, torch.empty(5, 0, device="cuda"), 32, torch.empty(1, 0, device="cuda"),
                   y)
    assert torch.all(y == 0)
    out = torch.full((0, 40), 1.0, device="cuda")
    sp.spmv_embed_q4(dc, ds, 32, torch.empty(0, dtype=torch.int64, device="cuda"), out)


# --- conversion ----------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 31), (5, 32), (3, 65), (17, 128), (4, 1000),
                                       (33, 129), (2, 4097), (64, 512), (1, 8192)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("w_type,scale_type,zeros", [
    ("f32", "f16", False), ("f32", "f32", True), ("bf16", "bf16", True), ("f16", "f16", False),
    ("bf16", "f32", False), ("f16", "bf16", True)])
def test_quantize_bit_for_bit(sp, rows, cols, group, w_type, scale_type, zeros):
    rng = np.random.default_rng(rows + cols)
    w = ot.round_to(rng.standard_normal((rows, cols)) * 0.02, w_type)
    if rows > 2:
        w[1] = 0  # a row of empty groups
        w[2] = np.abs(w[2])  # one sign only
    want_codes, want_scales, want_zeros = ot.q4_quantize(w, group, scale_type, zeros)
    groups = want_scales.shape[1]
    codes = torch.full((rows, (cols + 1) // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, groups), 9.0, dtype=TYPES[scale_type], device="cuda")
    z = torch.full((rows, groups), 99, dtype=torch.uint8, device="cuda") if zeros else None
    dw = dev(w, w_type)
    back = torch.empty_like(dw)
    sp.spmv_q4_quantize(dw, codes, scales, group, zeros=z, back=back)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    assert np.array_equal(host(scales), want_scales)
    if zeros:
        assert np.array_equal(z.cpu().numpy(), want_zeros)
    values = ot.q4_values(want_codes, want_scales, want_zeros, group, cols).astype(np.float32)
    assert np.array_equal(host(back), ot.round_to(values, w_type))
    # in place, and without the values
    sp.spmv_q4_quantize(dw, codes, scales, group, zeros=z)
    sp.spmv_q4_quantize(dw, codes, scales, group, zeros=z, back=dw)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    assert torch.equal(dw, back)


@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_strides(sp, zeros):
    rows, cols, group = 9, 77, 32
    w = np.random.default_rng(2).standard_normal((rows, cols)).astype(np.float32)
    want_codes, want_scales, want_zeros = ot.q4_quantize(w, group, "f32", zeros)
    dw = padded(rows, cols, torch.float32, 83, float("nan"))
    dw.copy_(dev(w))
    codes = padded(rows, 39, torch.uint8, 50, 0xEE)
    scales = padded(rows, 3, torch.float32, 5, 9.0)
    z = padded(rows, 3, torch.uint8, 7, 99) if zeros else None
    back = padded(rows, cols, torch.float32, 90, 5.0)
    sp.spmv_q4_quantize(dw, codes, scales, group, zeros=z, back=back)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    assert np.array_equal(host(scales), want_scales)
    assert torch.all(codes._base[:, 39:] == 0xEE) and torch.all(scales._base[:, 3:] == 9.0)
    assert torch.all(back._base[:, cols:] == 5.0)
    if zeros:
        assert np.array_equal(z.cpu().numpy(), want_zeros) and torch.all(z._base[:, 3:] == 99)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("w_type,scale_type", [("f32", "f32"), ("f32", "f16"), ("bf16", "bf16")])
def test_quantize_of_faulty_groups(sp, zeros, w_type, scale_type):
    """Infinities, NaN, overflowing and vanishing scales."""
    w = np.full((1, 256), 0.5, np.float32)
    w[0, 3] = np.inf
    w[0, 40] = np.nan
    w[0, 70] = -np.inf
    w[0, 96:128] = 1e-44 if w_type == "f32" else 0  # a scale below the least of its type
    w[0, 130] = 3e38  # overflows an fp16 scale
    w[0, 160:192] = 0
    w = ot.round_to(w, w_type)
    want_codes, want_scales, want_zeros = ot.q4_quantize(w, 32, scale_type, zeros)
    codes = torch.empty(1, 128, dtype=torch.uint8, device="cuda")
    scales = torch.empty(1, 8, dtype=TYPES[scale_type], device="cuda")
    z = torch.empty(1, 8, dtype=torch.uint8, device="cuda") if zeros else None
    back = torch.empty(1, 256, dtype=TYPES[w_type], device="cuda")
    sp.spmv_q4_quantize(dev(w, w_type), codes, scales, 32, zeros=z, back=back)
    assert np.array_equal(host(scales), want_scales, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    if zeros:
        assert np.array_equal(z.cpu().numpy(), want_zeros)
    fault = ~np.isfinite(want_scales[0]).repeat(32)
    got = host(back)[0]
    assert np.all(np.isnan(got[fault])) and np.all(np.isfinite(got[~fault]))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("w_type,scale_type", [("f32", "f32"), ("f32", "f16"), ("f16", "f16"),
                                               ("f16", "f32"), ("bf16", "bf16"),
                                               ("bf16", "f16")])
@pytest.mark.parametrize("cols,group", [(256, 32), (331, 32), (1160, 64), (333, 128), (1, 32)])
def test_quantize_of_faulty_groups_of_any_row(sp, cols, group, w_type, scale_type, zeros):
    """Infinities and NaN at the first and the last column, in the middle and in a partial
    last group, and scales that overflow or vanish, in rows of every alignment: exactly
    their groups have values that are NaN, the others are converted as ever."""
    large = {"f32": 3e38, "f16": 65504.0, "bf16": 3e38}[w_type]
    least = {"f32": 1e-44, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}[w_type]
    rng = np.random.default_rng(cols)
    w = rng.standard_normal((12, cols)).astype(np.float32)
    w[0, 0] = np.inf
    w[1, -1] = np.nan
    w[2, cols // 2] = -np.inf
    w[3] = np.nan
    w[4, cols // 2] = large  # its scale overflows fp16 where the weight is of more range
    w[5, cols // 2] = -large
    w[6] = least  # a scale below the least of its type, or subnormal
    w[7, ::3] = -large
    w[7, 1::3] = large  # with zero points the range itself overflows fp32
    w[8] = -least
    w[9, cols // 2:] = 0
    w[10, -1] = np.inf
    w[10, 0] = np.nan
    w = ot.round_to(w, w_type)
    want_codes, want_scales, want_zeros = ot.q4_quantize(w, group, scale_type, zeros)
    groups = want_scales.shape[1]
    codes = torch.empty(12, (cols + 1) // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(12, groups, dtype=TYPES[scale_type], device="cuda")
    z = torch.empty(12, groups, dtype=torch.uint8, device="cuda") if zeros else None
    back = torch.empty(12, cols, dtype=TYPES[w_type], device="cuda")
    sp.spmv_q4_quantize(dev(w, w_type), codes, scales, group, zeros=z, back=back)
    assert np.array_equal(host(scales), want_scales, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    if zeros:
        assert np.array_equal(z.cpu().numpy(), want_zeros)
    fault = ~np.isfinite(want_scales).repeat(group, 1)[:, :cols]
    got = host(back)
    assert np.all(np.isnan(got[fault])) and not np.any(np.isnan(got[~fault]))
    first, last = slice(0, group), slice((groups - 1) * group, cols)
    assert np.all(fault[0, first]) and np.all(fault[1, last]) and np.all(fault[3])
    assert not np.any(fault[0, group:]) and not np.any(fault[1, :(groups - 1) * group])


# --- rows back in dense form -----------------------------------------------------------------
@pytest.mark.parametrize("cols", [1, 31, 64, 100, 129, 1000, 4096])
@pytest.mark.parametrize("group,scale_type,zeros,out_type", [
    (32, "bf16", False, "bf16"), (64, "f16", True, "f32"), (128, "f32", True, "f16")])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_rows(sp, cols, group, scale_type, zeros, out_type, index):
    vocab = 50
    codes, scales, z = make(cols, vocab, cols, group, scale_type, zeros)
    dc, ds, dz = dev(codes), dev(scales, scale_type), None if z is None else dev(z)
    at = np.arange(cols) // group
    zero = 8 if z is None else z[:, at].astype(np.int64)
    exact = (ot.unpack(codes, cols) - zero).astype(np.float32) * scales[:, at]  # in fp32
    tokens = np.array([0, 49, 7, -1, 50, 7, 2 ** 31 - 1, -2 ** 31, 21])
    if index == torch.int64:
        tokens = np.append(tokens, [2 ** 32 + 3, -2 ** 40])
    out = torch.full((len(tokens), cols), 5.0, dtype=TYPES[out_type], device="cuda")
    sp.spmv_embed_q4(dc, ds, group, dev(tokens).to(index), out, scale=1.7, zeros=dz)
    assert np.array_equal(host(out), ot.embed(exact, tokens, 1.7, out_type))
    whole = torch.empty(vocab, cols, dtype=TYPES[out_type], device="cuda")
    sp.spmv_embed_q4(dc, ds, group, None, whole, zeros=dz)
    assert np.array_equal(host(whole), ot.round_to(exact, out_type))


def test_conversion_lookup_and_product_agree(sp):
    """quantize's values, the rows read back and a product with unit vectors
    are the same matrix."""
    w = dev(np.random.default_rng(8).standard_normal((48, 96)).astype(np.float32))
    codes = torch.empty(48, 48, dtype=torch.uint8, device="cuda")
    scales = torch.empty(48, 3, device="cuda")
    z = torch.empty(48, 3, dtype=torch.uint8, device="cuda")
    back, rows = torch.empty_like(w), torch.empty_like(w)
    sp.spmv_q4_quantize(w, codes, scales, 32, zeros=z, back=back)
    sp.spmv_embed_q4(codes, scales, 32, None, rows, zeros=z)
    assert torch.equal(rows, back)
    y = torch.empty(96, 48, device="cuda")
    sp.spmv_q4_run(codes, scales, 32, torch.eye(96, device="cuda"), y, zeros=z)
    assert torch.equal(y.t(), back)


# Products whose vectors a block takes into shared memory in several phases: (rows, columns,
# vectors, their type, group, zero points, bytes of padding to a row of codes, whether c is
# given, then the blocks that share a tile's columns; test_q4_plan.py asks for these and for
# the phases). With 8 blocks and 32 * 8 x more bytes than a block has they have no choice;
# the tall ones have several tiles to a block and more tiles than blocks.
PHASED = [(32, 200_000, 16, "bf16", 128, False, 0, False, 8),
          (32, 200_001, 16, "f16", 32, True, 0, True, 8),
          (2600, 80_003, 4, "f32", 64, True, 0, True, 8),
          (2600, 80_003, 4, "f32", 64, False, 14, False, 8),
          (80_327, 5880, 5, "f32", 128, False, 4, True, 2),
          (5647, 15_741, 16, "f16", 32, True, 0, False, 8),
          (124_910, 4029, 5, "f32", 32, True, 1, True, 1),
          (71_998, 1826, 16, "bf16", 64, True, 0, True, 1),
          (163_092, 2622, 13, "bf16", 128, False, 0, False, 1)]


def whole_product(codes, scales, zeros, group, x, c):
    """(y, sum of magnitudes) in 64 bits on the GPU, a block of rows at a time."""
    cols = x.shape[1]
    k = torch.arange(cols, device="cuda")
    xd = x.double()
    ys, mags = [], []
    for b in torch.arange(codes.shape[0], device="cuda").split(max(1, 2 ** 26 // cols)):
        q = codes[b][:, k // 2]
        a = torch.where(k % 2 == 0, q & 15, q >> 4).double()
        a -= 8.0 if zeros is None else zeros[b][:, k // group].double()
        a *= scales[b][:, k // group].double()
        ys.append(xd @ a.t())
        mags.append(xd.abs() @ a.abs().t())
    y, mag = torch.cat(ys, 1), torch.cat(mags, 1)
    return (y, mag) if c is None else (y + c.double(), mag + c.double().abs())


@pytest.mark.parametrize("rows,cols,n,x_type,group,zeros,pad,residual,blocks", PHASED)
def test_vectors_in_several_phases(sp, rows, cols, n, x_type, group, zeros, pad, residual,
                                   blocks):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    width, groups = (cols + 1) // 2, -(-cols // group)
    codes = torch.randint(0, 256, (rows, width + pad), device="cuda", generator=gen,
                          dtype=torch.uint8)[:, :width]
    scales = torch.rand(rows, groups, device="cuda", generator=gen).sub_(0.5).mul_(0.04)
    scales = scales.to(torch.bfloat16)
    z = (torch.randint(0, 16, (rows, groups), device="cuda", generator=gen, dtype=torch.uint8)
         if zeros else None)
    x = torch.randn(n, cols, device="cuda", generator=gen).to(TYPES[x_type])
    c = torch.randn(n, rows, device="cuda", generator=gen) if residual else None
    y = torch.full((n, rows), float("nan"), device="cuda")
    sp.spmv_q4_run(codes, scales, group, x, y, c=c, zeros=z)
    want, mag = whole_product(codes, scales, z, group, x, c)
    bound = (8 + groups + 32) * 2.0 ** -22 * mag
    bound = bound + (want.abs() + bound) * 2.0 ** -24 + 2.0 ** -150  # half a unit of fp32
    assert bool(((y.double() - want).abs() <= bound).all())
    again = torch.zeros_like(y) if c is None else c.clone()
    sp.spmv_q4_run(codes, scales, group, x, again, c=None if c is None else again, zeros=z)
    assert torch.equal(again, y)  # bit for bit, and in place


# --- streams, graphs, sizes ------------------------------------------------------------------
def test_on_another_stream_and_in_a_graph(sp):
    codes, scales, z = make(12, 300, 1024, 64, "f16", True)
    values = ot.q4_values(codes, scales, z, 64, 1024)
    x = ot.round_to(np.random.default_rng(5).standard_normal((2, 1024)), "f16")
    dc, ds, dz, dx = dev(codes), dev(scales, "f16"), dev(z), dev(x, "f16")
    y = torch.zeros(2, 300, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sp.spmv_q4_run(dc, ds, 64, dx, y, zeros=dz, stream=side)
    side.synchronize()
    check_product(host(y), values, x, None, 16, "f32")
    first = y.clone()
    out = torch.zeros(4, 1024, dtype=torch.float16, device="cuda")
    tokens = torch.tensor([3, 299, -1, 0], device="cuda")
    sp.spmv_embed_q4(dc, ds, 64, tokens, out, zeros=dz)
    rows = out.clone()
    y.zero_()
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sp.spmv_embed_q4(dc, ds, 64, tokens, out, zeros=dz)
        sp.spmv_q4_run(dc, ds, 64, dx, y, zeros=dz)
    torch.cuda.synchronize()
    assert torch.all(y == 0)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first) and torch.equal(out, rows)  # bit for bit, run after run


def test_offsets_past_32_bits(sp):
    """Codes of more than 2^31 bytes: the last rows are read from their own
    place, by the product and by the lookup."""
    rows, cols, group = 540_000, 8192, 128
    codes = torch.zeros(rows, cols // 2, dtype=torch.uint8, device="cuda")
    codes.fill_(0x88)
    scales = torch.ones(rows, cols // group, dtype=torch.bfloat16, device="cuda")
    assert codes.numel() > 2 ** 31
    tail, tail_scales, _ = make(13, 40, cols, group, "bf16", False)
    codes[-40:] = dev(tail)
    scales[-40:] = dev(tail_scales, "bf16")
    values = ot.q4_values(tail, tail_scales, None, group, cols)
    x = ot.round_to(np.random.default_rng(7).standard_normal((1, cols)), "bf16")
    y = torch.full((1, rows), 3.0, device="cuda")
    sp.spmv_q4_run(codes, scales, group, dev(x, "bf16"), y)
    assert torch.all(y[:, :-40] == 0)
    check_product(host(y[:, -40:]), values, x, None, cols // group, "f32")
    out = torch.empty(2, cols, device="cuda")
    sp.spmv_embed_q4(codes, scales, group, torch.tensor([rows - 1, rows - 40], device="cuda"), out)
    assert np.array_equal(host(out), values[[39, 0]].astype(np.float32))


@pytest.mark.parametrize("group", [32, 128])
def test_the_widest_row(sp, group):
    """As many columns as an int32 holds, in 1 GB of codes, with results from the columns
    at the two ends. The columns between have the value 0, so that their terms are exact
    and the bound is that of the few groups at the ends."""
    cols = 2 ** 31 - 1
    groups, tail = -(-cols // group), (cols // group - 2) * group
    codes = torch.full((1, (cols + 1) // 2), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.ones(1, groups, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(1, cols, dtype=torch.bfloat16, device="cuda")
    want, mag = np.zeros((1, 1)), np.zeros((1, 1))
    for seed, first in ((21, 0), (22, tail)):
        n = min(3 * group, cols - first)
        part, part_scales, _ = make(seed, 1, n, group, "bf16", False)
        v = ot.round_to(np.random.default_rng(seed).standard_normal((1, n)), "bf16")
        codes[:, first // 2:first // 2 + part.shape[1]] = dev(part)
        scales[:, first // group:first // group + part_scales.shape[1]] = dev(part_scales, "bf16")
        x[:, first:first + n] = dev(v, "bf16")
        y, m = ot.q4_run(ot.q4_values(part, part_scales, None, group, n), v)
        want, mag = want + y, mag + m
    y = torch.full((1, 1), 7.0, device="cuda")
    sp.spmv_q4_run(codes, scales, group, x, y)
    bound = (8 + 6 + 32) * 2.0 ** -22 * mag + ot.half_ulp(np.abs(want), "f32")
    assert abs(host(y)[0, 0] - want[0, 0]) <= bound[0, 0]
    assert abs(want[0, 0]) > 100 * bound[0, 0]  # y = 0 fails


def test_fp32_vectors_come_back_bit_for_bit(sp):
    """The unit matrix times vectors of every finite exponent, subnormal ones among them."""
    rng = np.random.default_rng(17)
    bits = rng.integers(0, 2 ** 32, (70, 32), dtype=np.uint64).astype(np.uint32)
    bits[:10] &= 0x807FFFFF  # subnormal
    bits[10:30] = (bits[10:30] & 0x807FFFFF) | (rng.integers(1, 24, (20, 32)) << 23).astype(
        np.uint32)
    bits[30, :5] = [0, 0x80000000, 1, 0x7F7FFFFF, 0x00800000]
    x = bits.view(np.float32)
    x[~np.isfinite(x)] = 1.5
    codes = ot.pack(np.full((32, 32), 8, np.uint8) + np.eye(32, dtype=np.uint8))
    y = torch.empty(70, 32, device="cuda")
    sp.spmv_q4_run(dev(codes), torch.ones(32, 1, device="cuda"), 32, dev(x), y)
    assert np.array_equal(host(y), x)


@pytest.mark.parametrize("x_type,scale", [("f32", 1e-36), ("f32", 1e-37), ("f32", 1e-38),
                                          ("f32", 1e-40), ("f32", 1e-42), ("bf16", 1e-37),
                                          ("bf16", 1e-39)])
def test_tiny_vectors(sp, x_type, scale):
    """Within the stated bound, whose absolute term (a rounding to a multiple of 2^-149 for
    each group's sum and each partial sum's three parts) is far below the results."""
    rows, cols, group = 40, 333, 32
    codes, scales, z = make(15, rows, cols, group, "f32", True)
    scales *= 50
    x = ot.round_to((np.random.default_rng(16).standard_normal((3, cols)) * scale)
                    .astype(np.float32), x_type)
    want, mag = ot.q4_run(ot.q4_values(codes, scales, z, group, cols), x)
    y = torch.zeros(3, rows, device="cuda")
    sp.spmv_q4_run(dev(codes), dev(scales), group, dev(x, x_type), y, zeros=dev(z))
    bound = (40 + scales.shape[1]) * (2.0 ** -22 * mag + 2.0 ** -148)
    assert np.all(np.abs(host(y).astype(np.float64) - want) <= bound)
    assert np.all(bound < mag / 50) and np.mean(np.abs(want) > bound) > 0.9  # y = 0 fails


# --- refusals ----------------------------------------------------------------------------------
def test_refusals(sp):
    import ctypes as C
    codes, scales, z = make(14, 8, 64, 32, "f32", True)
    dc, ds, dz = dev(codes), dev(scales), dev(z)
    x, y = torch.zeros(2, 64, device="cuda"), torch.zeros(2, 8, device="cuda")

    def code_of(call):
        with pytest.raises(sp.SpmvError) as e:
            call()
        return e.value.code

    bad = sp.SPMV_ERR_INVALID_ARG
    assert code_of(lambda: sp.spmv_q4_run(dc, ds, 16, x, y)) == bad  # group
    assert code_of(lambda: sp.spmv_q4_run(dc, ds, 48, x, y)) == bad
    both = torch.zeros(2, 80, device="cuda")
    assert code_of(lambda: sp.spmv_q4_run(dc, ds, 32, both[:, :64], both[:, 60:68])) == bad
    shared = torch.zeros(3, 8, device="cuda")  # c one row off y
    assert code_of(lambda: sp.spmv_q4_run(dc, ds, 32, x, shared[:2], c=shared[1:])) == bad
    w = torch.zeros(8, 64, device="cuda")
    assert code_of(lambda: sp.spmv_q4_quantize(w, w.view(torch.uint8)[:, :32], ds, 32)) == bad
    with pytest.raises(TypeError):
        sp.spmv_q4_run(dc, ds, 32, x.double(), y)
    with pytest.raises(ValueError):
        sp.spmv_q4_run(dc, ds, 32, x, y[:1])
    with pytest.raises(ValueError):
        sp.spmv_q4_run(dc, ds[:, :1], 32, x, y)
    with pytest.raises(ValueError):
        sp.spmv_q4_run(dc, ds, 32, x.cpu(), y)
    with pytest.raises(ValueError):
        sp.spmv_q4_run(dc, ds, 32, torch.zeros(64, 2, device="cuda").t(), y)
    # a host pointer and a pointer off an element's size reach the C call
    a = sp.spmv_q4(8, 64, 32, sp.SPMV_F32, dc.data_ptr(), 32, ds.data_ptr(), 2, None, 0)
    hostx = np.zeros((2, 64), np.float32)

    def run(xp, yp, n=2, ldx=64, ldy=8):
        return sp._lib.spmv_q4_run(C.byref(a), n, sp.SPMV_F32, xp, ldx, None, 0, sp.SPMV_F32, yp,
                                   ldy, None)

    assert run(hostx.ctypes.data, y.data_ptr()) == bad
    assert run(x.data_ptr() + 2, y.data_ptr()) == bad
    assert run(x.data_ptr(), y.data_ptr(), ldx=63) == bad
    assert run(x.data_ptr(), y.data_ptr(), ldy=7) == bad
    assert run(x.data_ptr(), y.data_ptr(), n=-1) == bad
    assert run(x.data_ptr(), y.data_ptr()) == sp.SPMV_OK
    out = torch.zeros(9, 64, device="cuda")
    assert sp._lib.spmv_embed_q4(C.byref(a), 9, 4, None, 1.0, sp.SPMV_F32, out.data_ptr(), 64,
                                 None) == bad  # nine rows of eight
    torch.cuda.synchronize()
