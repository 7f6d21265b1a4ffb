"""Token lookups (bit for bit) and their gradient against the 64-bit
references.

Bound of a gradient entry with m terms: sums of at most 32 terms, joined by
at most m/32 further additions, one product with the scale and, where it is
added to a table, one more addition: (min(m, 32) + m/32 + 4) * 2^-24 * the sum
of magnitudes, then half a unit of the result's type."""
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


# --- lookup ------------------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [1, 7, 8, 24, 100, 128, 1000, 4096])
@pytest.mark.parametrize("table_type,out_type", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"),
                                                 ("bf16", "bf16"), ("bf16", "f32"),
                                                 ("f16", "bf16")])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_lookup(sp, dim, table_type, out_type, index):
    vocab = 61
    rng = np.random.default_rng(dim)
    table = ot.round_to(rng.standard_normal((vocab, dim)), table_type)
    for n in (1, 2, 37):
        tokens = rng.integers(-3, vocab + 3, n)
        tokens[-1] = vocab - 1
        out = torch.full((n, dim), 5.0, dtype=TYPES[out_type], device="cuda")
        sp.spmv_embed(dev(table, table_type), dev(tokens).to(index), out, scale=3.3)
        assert np.array_equal(host(out), ot.embed(table, tokens, 3.3, out_type))


def test_lookup_of_far_tokens_and_faulty_rows(sp):
    """Tokens far outside the table read nothing; a NaN or an infinity stays
    in its own row."""
    table = np.ones((10, 16), np.float32)
    table[3] = np.nan
    table[4] = np.inf
    tokens = np.array([2 ** 40, -2 ** 40, 2 ** 32 + 1, 10, -1, 0, 3, 4, 9])
    out = torch.empty(len(tokens), 16, device="cuda")
    sp.spmv_embed(dev(table), dev(tokens), out)
    got = host(out)
    assert np.all(got[:5] == 0) and np.all(got[[5, 8]] == 1)
    assert np.all(np.isnan(got[6])) and np.all(np.isinf(got[7]))


@pytest.mark.parametrize("pad", [0, 1, 4, 8])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_lookup_strides(sp, pad, shift):
    vocab, dim, n = 20, 72, 13
    rng = np.random.default_rng(pad)
    table = ot.round_to(rng.standard_normal((vocab, dim)), "bf16")
    flat = torch.full((shift + vocab * (dim + pad),), float("nan"), dtype=torch.bfloat16,
                      device="cuda")
    dt = flat[shift:].view(vocab, dim + pad)[:, :dim]
    dt.copy_(dev(table))
    oflat = torch.full((shift + n * (dim + pad),), 7.0, dtype=torch.bfloat16, device="cuda")
    out = oflat[shift:].view(n, dim + pad)[:, :dim]
    tokens = rng.integers(0, vocab, n)
    sp.spmv_embed(dt, dev(tokens), out, scale=0.5)
    assert np.array_equal(host(out), ot.embed(table, tokens, 0.5, "bf16"))
    gaps = torch.ones(oflat.numel(), dtype=torch.bool, device="cuda")
    gaps[shift:].view(n, dim + pad)[:, :dim] = False
    assert torch.all(oflat[gaps] == 7.0)


# --- gradient ------------------------------------------------------------------------------------
def check_grad(got, g, tokens, vocab, scale, out_type, base=None):
    want, mag, m = ot.embed_grad(g, tokens, vocab, scale, base)
    bound = (np.minimum(m, 32) + m / 32 + 4)[:, None] * 2.0 ** -24 * mag
    bound = bound + ot.half_ulp(np.abs(want) + bound, out_type)
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(err <= bound), float((err / bound).max())
    if base is None:
        assert np.all(got[m == 0] == 0)
    else:
        assert np.array_equal(got[m == 0], base[m == 0])


def tokens_of(kind, n, vocab, rng):
    if kind == "uniform":
        return rng.integers(0, vocab, n)
    if kind == "skewed":
        return np.minimum((vocab ** rng.random(n)).astype(np.int64) - 1, vocab - 1)
    if kind == "one":
        return np.full(n, vocab // 2)
    if kind == "none":
        return np.full(n, -1)
    if kind == "ends":  # the first and the last row only, with padding between
        return rng.choice([0, vocab - 1, -1, vocab], n)
    raise ValueError(kind)


@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "none", "ends"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 100, 1023, 4097])
@pytest.mark.parametrize("g_type,out_type,dim,vocab", [
    ("f32", "f32", 8, 300), ("bf16", "f32", 100, 5), ("bf16", "bf16", 64, 1000),
    ("f16", "f16", 33, 129), ("f16", "f32", 256, 70000), ("f32", "bf16", 1, 1)])
def test_gradient(sp, kind, n, g_type, out_type, dim, vocab):
    rng = np.random.default_rng(n)
    tokens = tokens_of(kind, n, vocab, rng)
    g = ot.round_to(rng.standard_normal((n, dim)), g_type)
    dt = torch.full((vocab, dim), float("nan"), dtype=TYPES[out_type], device="cuda")
    sp.spmv_embed_grad(dev(g, g_type), dev(tokens), dt, scale=1.5)
    check_grad(host(dt), g, tokens, vocab, 1.5, out_type)
    base = ot.round_to(rng.standard_normal((vocab, dim)), out_type)
    dt = dev(base, out_type)
    sp.spmv_embed_grad(dev(g, g_type), dev(tokens).to(torch.int32), dt, scale=-0.5,
                       accumulate=True)
    check_grad(host(dt), g, tokens, vocab, -0.5, out_type, base)


@pytest.mark.parametrize("terms", ["equal", "positive", "mixed"])
@pytest.mark.parametrize("n,vocab,dim,g_type", [(4097, 1000, 256, "f32"), (19_000, 9, 256, "f32"),
                                                (19_000, 40_000, 300, "bf16"),
                                                (60_000, 2, 64, "f32"), (70_000, 5, 33, "f16"),
                                                (3000, 7, 1000, "bf16")])
def test_long_rows_of_terms_of_one_sign(sp, terms, n, vocab, dim, g_type):
    """Most tokens are one, and the errors of its sum do not cancel. The chain of additions
    behind a row of m terms, whatever the split: up to 32 in a chunk (twice that where a
    row ends in the next one); a partial sum for each 4 terms at least, added in 4
    groups at least, so m / 16 at most; 8 for joining the groups; the first chunk's sum,
    the scale and the table's own value: (64 + m / 16 + 12) * 2^-24 of the magnitudes."""
    rng = np.random.default_rng(n)
    tokens = np.full(n, vocab // 2)
    tokens[::50] = rng.integers(0, vocab, len(tokens[::50]))
    g = {"equal": lambda: np.full((n, dim), 0.1), "positive": lambda: rng.random((n, dim)),
         "mixed": lambda: rng.standard_normal((n, dim))}[terms]()
    g = ot.round_to(g.astype(np.float32), g_type)
    base = rng.random((vocab, dim)).astype(np.float32)
    for add in (False, True):
        dt = dev(base)
        sp.spmv_embed_grad(dev(g, g_type), dev(tokens), dt, scale=0.3, accumulate=add)
        want, mag, m = ot.embed_grad(g, tokens, vocab, float(np.float32(0.3)),
                                     base if add else None)
        bound = (np.minimum(m, 64) + m / 16 + 12)[:, None] * 2.0 ** -24 * mag
        err = np.abs(host(dt).astype(np.float64) - want)
        assert np.all(err <= bound + 2.0 ** -150), float((err / bound).max())
        assert np.all(bound <= 3e-4 * mag)  # a term of ten thousand that is missing shows


@pytest.mark.parametrize("n,vocab,kind", [(65536, 50000, "skewed"), (65537, 200, "uniform"),
                                          (70001, 300_000, "skewed"), (200_000, 3, "uniform"),
                                          (40_000, 131072, "one"), (16384, 2 ** 18 + 1, "ends")])
def test_gradient_of_many_tokens(sp, n, vocab, kind):
    rng = np.random.default_rng(n)
    tokens = tokens_of(kind, n, vocab, rng)
    dim = 16
    g = ot.round_to(rng.standard_normal((n, dim)), "bf16")
    dt = torch.full((vocab, dim), float("nan"), device="cuda")
    sp.spmv_embed_grad(dev(g, "bf16"), dev(tokens), dt)
    check_grad(host(dt), g, tokens, vocab, 1.0, "f32")
    again = torch.full((vocab, dim), float("nan"), device="cuda")
    sp.spmv_embed_grad(dev(g, "bf16"), dev(tokens), again)
    assert torch.equal(dt, again)  # bit for bit


@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "ends"])
@pytest.mark.parametrize("n", [127, 128, 129, 2047, 2048, 2049, 4096, 8192, 8193, 20000])
def test_gradient_where_the_way_of_sorting_changes(sp, kind, n):
    """Lengths around those at which tokens are sorted another way; vocabulary
    numbers up to the largest and 64-bit tokens that wrap around to small ones."""
    rng = np.random.default_rng(n)
    vocab, dim = 2 ** 18 + 3, 8
    tokens = tokens_of(kind, n, vocab, rng)
    tokens[::97] = 2 ** 32 + 1
    tokens[50::97] = -2 ** 63
    g = ot.round_to(rng.standard_normal((n, dim)), "f16")
    base = rng.standard_normal((vocab, dim)).astype(np.float32)
    dt = dev(base, "f32")
    sp.spmv_embed_grad(dev(g, "f16"), dev(tokens), dt, scale=2.0, accumulate=True)
    check_grad(host(dt), g, tokens, vocab, 2.0, "f32", base)
    again = dev(base, "f32")
    sp.spmv_embed_grad(dev(g, "f16"), dev(tokens), again, scale=2.0, accumulate=True)
    assert torch.equal(dt, again)  # bit for bit


@pytest.mark.parametrize("n,vocab,kind", [(65537, 131072, "skewed"), (131072, 50257, "uniform"),
                                          (131073, 50257, "uniform"), (100_000, 7, "ends")])
def test_gradient_of_tokens_beyond_a_cluster(sp, n, vocab, kind):
    rng = np.random.default_rng(n)
    tokens = tokens_of(kind, n, vocab, rng)
    g = ot.round_to(rng.standard_normal((n, 8)), "bf16")
    dt = torch.full((vocab, 8), float("nan"), device="cuda")
    sp.spmv_embed_grad(dev(g, "bf16"), dev(tokens), dt)
    check_grad(host(dt), g, tokens, vocab, 1.0, "f32")


@pytest.mark.parametrize("g_type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("table_type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,pad,shift", [(4, 0, 0), (12, 0, 0), (300, 0, 4), (60, 4, 0),
                                           (1028, 0, 0), (64, 4, 4), (64, 2, 0), (64, 0, 2),
                                           (2052, 8, 8)])
def test_rows_on_part_of_a_16_byte_boundary(sp, dim, pad, shift, g_type, table_type):
    """Rows whose lengths, starts and distances allow 4 elements at a time, or
    just fail to: lookup, and gradient written and added to."""
    rng = np.random.default_rng(dim + pad + shift)
    vocab, n = 40, 150

    def rows(m, kind, a=None):
        flat = torch.full((shift + m * (dim + pad),), 7.0, dtype=TYPES[kind], device="cuda")
        t = flat[shift:].view(m, dim + pad)[:, :dim]
        if a is not None:
            t.copy_(dev(a))
        return flat, t

    def untouched(flat, m):
        gaps = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
        gaps[shift:].view(m, dim + pad)[:, :dim] = False
        return bool(torch.all(flat[gaps] == 7.0))

    tokens = rng.integers(-2, vocab, n)
    tokens[:70] = 3
    table = ot.round_to(rng.standard_normal((vocab, dim)), table_type)
    g = ot.round_to(rng.standard_normal((n, dim)), g_type)
    flat, out = rows(n, g_type)
    sp.spmv_embed(rows(vocab, table_type, table)[1], dev(tokens), out, scale=0.7)
    assert np.array_equal(host(out), ot.embed(table, tokens, 0.7, g_type))
    assert untouched(flat, n)
    for add in (False, True):
        flat, dt = rows(vocab, table_type, table)
        sp.spmv_embed_grad(rows(n, g_type, g)[1], dev(tokens), dt, scale=1.5, accumulate=add)
        check_grad(host(dt), g, tokens, vocab, 1.5, table_type, table if add else None)
        assert untouched(flat, vocab)


def test_gradient_ignores_what_padding_holds(sp):
    """NaN and infinities in the rows of tokens outside the table, and in the
    gaps between rows, reach nothing."""
    rng = np.random.default_rng(1)
    n, dim, vocab = 200, 40, 30
    tokens = rng.integers(0, vocab, n)
    tokens[::7] = -1
    tokens[3::11] = vocab
    g = rng.standard_normal((n, dim)).astype(np.float32)
    outside = (tokens < 0) | (tokens >= vocab)
    big = torch.full((n, dim + 8), float("nan"), device="cuda")
    big[:, :dim] = dev(g)
    big[dev(outside), :dim] = float("inf")
    flat = torch.full((vocab, dim + 8), 9.0, device="cuda")
    sp.spmv_embed_grad(big[:, :dim], dev(tokens), flat[:, :dim], scale=2.0)
    g[outside] = 0
    check_grad(host(flat[:, :dim]), g, tokens, vocab, 2.0, "f32")
    assert torch.all(flat[:, dim:] == 9.0)


def test_gradient_with_a_nan_stays_in_its_row(sp):
    g = np.ones((100, 8), np.float32)
    tokens = np.arange(100) % 10
    g[33] = np.nan
    dt = torch.empty(12, 8, device="cuda")
    sp.spmv_embed_grad(dev(g), dev(tokens), dt)
    got = host(dt)
    assert np.all(np.isnan(got[3])) and np.all(got[10:] == 0)
    assert np.all(got[[0, 1, 2, 4, 5, 6, 7, 8, 9]] == 10)


def test_gradient_against_differences(sp):
    """L(T) = sum of w * lookup(T) is linear in T: its difference quotient
    along a direction is the gradient's product with it."""
    rng = np.random.default_rng(4)
    vocab, dim, n = 40, 24, 300
    tokens = rng.integers(-2, vocab, n)
    table = rng.standard_normal((vocab, dim)).astype(np.float32)
    w = rng.standard_normal((n, dim)).astype(np.float32)
    dt = torch.empty(vocab, dim, device="cuda")
    sp.spmv_embed_grad(dev(w), dev(tokens), dt, scale=4.0)
    grad = dt.double().cpu().numpy()

    def loss(t):
        out = torch.empty(n, dim, device="cuda")
        sp.spmv_embed(dev(t.astype(np.float32)), dev(tokens), out, scale=4.0)
        return float((out.double().cpu().numpy() * w).sum())

    h = 0.25
    for _ in range(5):
        d = rng.choice([-1.0, 0.0, 1.0], table.shape)
        slope = (loss(table + h * d) - loss(table - h * d)) / (2 * h)
        # each lookup rounds its sum and product (2 * 2^-24 of 4 * 2 * |t| * |w|), over 2h
        slack = 2 * 2.0 ** -24 * 4 * 3 * 4.5 * np.abs(w).sum() / (2 * h)
        assert abs(slope - (grad * d).sum()) <= slack


def test_gradient_over_nothing(sp):
    dt = torch.full((6, 4), 3.0, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    sp.spmv_embed_grad(torch.empty(0, 4, device="cuda"), none, dt, accumulate=True)
    assert torch.all(dt == 3.0)
    sp.spmv_embed_grad(torch.empty(0, 4, device="cuda"), none, dt)
    assert torch.all(dt == 0.0)


def test_lookup_and_gradient_on_another_stream_and_in_a_graph(sp):
    rng = np.random.default_rng(6)
    n, vocab, dim = 3000, 500, 64
    tokens = tokens_of("skewed", n, vocab, rng)
    g = rng.standard_normal((n, dim)).astype(np.float32)
    dg, dk = dev(g), dev(tokens)
    dt = torch.zeros(vocab, dim, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sp.spmv_embed_grad(dg, dk, dt, stream=side)
    side.synchronize()
    check_grad(host(dt), g, tokens, vocab, 1.0, "f32")
    first = dt.clone()
    work = torch.empty(sp.spmv_embed_grad_workspace(vocab, dim, n), dtype=torch.uint8,
                       device="cuda")
    out = torch.zeros(n, dim, device="cuda")
    sp.spmv_embed(dt, dk, out)
    sp.spmv_embed_grad(dg, dk, dt, workspace=work)
    torch.cuda.synchronize()
    dt.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.spmv_embed_grad(dg, dk, dt, workspace=work)
        sp.spmv_embed(dt, dk, out)
    torch.cuda.synchronize()
    assert torch.all(dt == 0)
    for _ in range(2):
        work.fill_(0xFF)  # nothing is kept in the workspace
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dt, first)
        assert torch.equal(out, first[dk])


@pytest.fixture(params=["direct", "public"])
def scratch(request, sp, monkeypatch):
    """Scratch by either way of asking torch for it."""
    if request.param == "public":
        monkeypatch.setattr(sp, "_take_scratch", sp._public_take)
        monkeypatch.setattr(sp, "_free_scratch", sp._public_free)


def test_scratch_of_its_own_in_a_graph(sp, scratch):
    """Two gradients captured with no workspace given; what is allocated and written
    between the replays reaches neither."""
    rng = np.random.default_rng(3)
    n, vocab, dim = 3000, 400, 64
    tokens = rng.integers(-1, vocab, n)
    dg, dk = dev(rng.standard_normal((n, dim)).astype(np.float32)), dev(tokens)
    one, two = torch.empty(vocab, dim, device="cuda"), torch.empty(vocab, dim, device="cuda")
    sp.spmv_embed_grad(dg, dk, one)
    check_grad(host(one), host(dg), tokens, vocab, 1.0, "f32")
    want = one.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.spmv_embed_grad(dg, dk, one)
        sp.spmv_embed_grad(dg, dk, two, scale=2.0)
    size = sp.spmv_embed_grad_workspace(vocab, dim, n)
    for _ in range(3):
        one.zero_()
        two.zero_()
        other = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        graph.replay()
        other += [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert torch.equal(one, want) and torch.equal(two, 2 * want)


def test_scratch_of_its_own_beside_other_work(sp, scratch):
    """Gradients on a stream that is behind (a large product is ahead of them there),
    while another stream takes memory of the scratch's size and writes it."""
    rng = np.random.default_rng(4)
    n, vocab, dim = 5000, 300, 64
    tokens = rng.integers(-1, vocab, n)
    dg, dk = dev(rng.standard_normal((n, dim)).astype(np.float32)), dev(tokens)
    outs = [torch.empty(vocab, dim, device="cuda") for _ in range(4)]
    sp.spmv_embed_grad(dg, dk, outs[0])
    check_grad(host(outs[0]), host(dg), tokens, vocab, 1.0, "f32")
    want = outs[0].clone()
    size = sp.spmv_embed_grad_workspace(vocab, dim, n)
    a = torch.ones(4096, 4096, device="cuda")
    b = torch.empty_like(a)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(a, a, out=b)
        for i, o in enumerate(outs):
            if i % 2:
                sp.spmv_embed_grad(dg, dk, o, stream=side)
            else:
                with torch.cuda.stream(side):
                    sp.spmv_embed_grad(dg, dk, o)
            torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_offsets_past_32_bits(sp):
    """A table of more than 2^31 elements: lookups from and gradients into its
    last rows."""
    vocab, dim = 530_000, 4096
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    assert table.numel() > 2 ** 31
    table[-1] = 2.0
    table[-3] = 5.0
    tokens = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 1], device="cuda")
    out = torch.empty(4, dim, dtype=torch.bfloat16, device="cuda")
    sp.spmv_embed(table, tokens, out)
    assert [float(v) for v in out[:, 0]] == [2, 0, 5, 2]
    assert torch.equal(out, out[:, :1].expand(4, dim))
    sp.spmv_embed_grad(torch.ones(4, dim, dtype=torch.bfloat16, device="cuda"), tokens, table,
                       accumulate=True)
    assert torch.all(table[-1] == 4) and torch.all(table[-3] == 6) and torch.all(table[0] == 1)
    table.fill_(7.0)
    sp.spmv_embed_grad(torch.ones(4, dim, dtype=torch.bfloat16, device="cuda"), tokens, table)
    assert torch.all(table[-1] == 2) and torch.all(table[-3] == 1) and torch.all(table[0] == 1)
    assert not torch.any(table[1:-3]) and not torch.any(table[-2])


def test_refusals(sp):
    import ctypes as C
    bad = sp.SPMV_ERR_INVALID_ARG
    table = torch.zeros(10, 16, device="cuda")
    tokens = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.zeros(4, 16, device="cuda")

    def code_of(call):
        with pytest.raises(sp.SpmvError) as e:
            call()
        return e.value.code

    assert code_of(lambda: sp.spmv_embed(table, tokens, table[2:6])) == bad  # overlap
    assert code_of(lambda: sp.spmv_embed_grad(table[:4], tokens, table)) == bad
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    assert code_of(lambda: sp.spmv_embed_grad(out, tokens, table, workspace=small)) == bad
    with pytest.raises(ValueError):
        sp.spmv_embed(table, tokens, out[:3])
    with pytest.raises(ValueError):
        sp.spmv_embed(table, tokens, torch.zeros(4, 8, device="cuda"))
    with pytest.raises(TypeError):
        sp.spmv_embed(table, tokens.float(), out)
    with pytest.raises(ValueError):
        sp.spmv_embed(table, tokens.cpu(), out)
    lib = sp._lib

    def embed(tp=table.data_ptr(), index=4, kp=tokens.data_ptr(), ldt=16, ot_=0, tt=0, vocab=10):
        return lib.spmv_embed(vocab, 16, tt, tp, ldt, 4, index, kp, 1.0, ot_, out.data_ptr(), 16,
                              None)

    hosted = np.zeros(4, np.int32)
    assert embed() == sp.SPMV_OK
    for kw in (dict(index=2), dict(tt=3), dict(ot_=-1), dict(ldt=15), dict(vocab=-1),
               dict(tp=None), dict(tp=table.data_ptr() + 1), dict(kp=tokens.data_ptr() + 2),
               dict(kp=hosted.ctypes.data)):
        assert embed(**kw) == bad, kw
    b = C.c_int64()
    assert lib.spmv_embed_grad_workspace(10, 16, 4, None) == bad
    assert lib.spmv_embed_grad_workspace(-1, 16, 4, C.byref(b)) == bad
    torch.cuda.synchronize()
