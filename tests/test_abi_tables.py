"""The dense-table operators' C entries: exported, bound under their names, and
answering bad arguments before any CUDA call (no GPU needed)."""
import ctypes as C
import re
import os

import pytest
import torch

from conftest import ROOT

NAMES = ["spmv_q4_quantize", "spmv_q4_run", "spmv_embed", "spmv_embed_q4", "spmv_embed_grad",
         "spmv_embed_grad_workspace"]


@pytest.fixture(scope="module")
def sp():
    from conftest import build_library
    build_library()
    import spmv_sparse_storage_gb300 as sp
    return sp


def test_declared_exported_and_bound(sp):
    header = open(os.path.join(ROOT, "include", "spmv.h")).read()
    lib = C.CDLL(sp.LIB_PATH)
    for name in NAMES:
        assert re.search(rf"\bint {name}\(", header), name
        assert hasattr(lib, name) and callable(getattr(sp, name)) and name in sp.__all__
    assert sp.DTYPES == {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def q4(sp, rows=4, cols=64, group=32, scale_type=0, codes=4096, ld_codes=32, scales=4096,
       ld_scales=2, zeros=None, ld_zeros=0):
    return sp.spmv_q4(rows, cols, group, scale_type, codes, ld_codes, scales, ld_scales, zeros,
                      ld_zeros)


BAD_Q4 = [dict(rows=-1), dict(cols=-1), dict(group=0), dict(group=16), dict(group=96),
          dict(group=256), dict(scale_type=3), dict(scale_type=-1), dict(ld_codes=31),
          dict(ld_scales=1), dict(zeros=4096, ld_zeros=1), dict(codes=None), dict(scales=None),
          dict(scales=4098)]


@pytest.mark.parametrize("bad", BAD_Q4)
def test_bad_matrices(sp, bad):
    a = C.byref(q4(sp, **bad))
    p, lib, inv = 1 << 20, sp._lib, sp.SPMV_ERR_INVALID_ARG
    assert lib.spmv_q4_run(a, 1, 0, p, 64, None, 0, 0, p + 4096, 4, None) == inv
    assert lib.spmv_q4_quantize(a, 0, p, 64, None, 0, None) == inv
    assert lib.spmv_embed_q4(a, 1, 4, p, 1.0, 0, p + 4096, 64, None) == inv


def test_null_matrix(sp):
    lib, inv = sp._lib, sp.SPMV_ERR_INVALID_ARG
    assert lib.spmv_q4_run(None, 1, 0, 64, 64, None, 0, 0, 64, 4, None) == inv
    assert lib.spmv_q4_quantize(None, 0, 64, 64, None, 0, None) == inv
    assert lib.spmv_embed_q4(None, 1, 4, 64, 1.0, 0, 64, 64, None) == inv


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(xt=3), dict(yt=-1), dict(ldx=63), dict(ldy=3), dict(x=None), dict(y=None),
    dict(x=(1 << 20) + 2), dict(y=(1 << 21) + 2), dict(c=1 << 22, ldc=3), dict(c=(1 << 22) + 1),
    dict(x=1 << 21), dict(c=(1 << 21) + 8), dict(c=1 << 21, ldc=5, n=2), dict(y=4096)])
def test_bad_products(sp, bad):
    """Among them: y over x, c over y but not y itself, y over the codes."""
    a = dict(n=1, xt=0, x=1 << 20, ldx=64, c=None, ldc=4, yt=0, y=1 << 21, ldy=4)
    a.update(bad)
    m = q4(sp)
    assert sp._lib.spmv_q4_run(C.byref(m), a["n"], a["xt"], a["x"], a["ldx"], a["c"], a["ldc"],
                               a["yt"], a["y"], a["ldy"], None) == sp.SPMV_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(wt=5), dict(ldw=63), dict(w=None), dict(w=(1 << 20) + 1),
                                 dict(back=1 << 21, ldb=63), dict(back=(1 << 20) + 4),
                                 dict(back=1 << 20, ldb=65), dict(w=4096)])
def test_bad_conversions(sp, bad):
    """Among them: the values over W but not W itself, W over the codes."""
    a = dict(wt=0, w=1 << 20, ldw=64, back=None, ldb=64)
    a.update(bad)
    m = q4(sp, scales=8192)
    assert sp._lib.spmv_q4_quantize(C.byref(m), a["wt"], a["w"], a["ldw"], a["back"], a["ldb"],
                                    None) == sp.SPMV_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(vocab=-1), dict(dim=-1), dict(n=-1), dict(tt=3), dict(ot=3), dict(index=1),
    dict(table=None), dict(tokens=None), dict(out=None), dict(ldt=15), dict(ldo=15),
    dict(table=(1 << 20) + 2), dict(tokens=(1 << 21) + 2), dict(out=(1 << 22) + 1),
    dict(out=1 << 20), dict(out=1 << 21)])
def test_bad_lookups(sp, bad):
    a = dict(vocab=10, dim=16, tt=0, table=1 << 20, ldt=16, n=4, index=4, tokens=1 << 21, ot=0,
             out=1 << 22, ldo=16)
    a.update(bad)
    assert sp._lib.spmv_embed(a["vocab"], a["dim"], a["tt"], a["table"], a["ldt"], a["n"],
                              a["index"], a["tokens"], 1.0, a["ot"], a["out"], a["ldo"],
                              None) == sp.SPMV_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(vocab=-1), dict(dim=-1), dict(n=-1), dict(gt=3), dict(tt=3), dict(index=3),
    dict(add=2), dict(g=None), dict(tokens=None), dict(dt=None), dict(work=None), dict(ldg=15),
    dict(ldd=15), dict(bytes=-1), dict(bytes=16), dict(work=(1 << 24) + 8), dict(g=1 << 23),
    dict(work=1 << 23), dict(tokens=1 << 23), dict(g=(1 << 20) + 2)])
def test_bad_gradients(sp, bad):
    """Among them: g, the tokens or the workspace over the gradient."""
    a = dict(vocab=10, dim=16, gt=0, g=1 << 20, ldg=16, n=4, index=4, tokens=1 << 22, add=0,
             tt=0, dt=1 << 23, ldd=16, work=1 << 24, bytes=1 << 20)
    a.update(bad)
    assert sp._lib.spmv_embed_grad(
        a["vocab"], a["dim"], a["gt"], a["g"], a["ldg"], a["n"], a["index"], a["tokens"], 1.0,
        a["add"], a["tt"], a["dt"], a["ldd"], a["work"], a["bytes"],
        None) == sp.SPMV_ERR_INVALID_ARG


def test_workspace_sizes(sp):
    assert sp.spmv_embed_grad_workspace(100, 64, 0) == 0
    assert sp.spmv_embed_grad_workspace(0, 64, 10) == 0
    sizes = [sp.spmv_embed_grad_workspace(1000, 256, n) for n in (1, 100, 10_000, 65536, 65537,
                                                                  1_000_000)]
    assert all(s > 0 for s in sizes)
    # the partial sums: two rows of fp32 for each 4 tokens at most, and the sort's 16 + bytes
    for n, s in zip((1, 100, 10_000, 65536, 65537, 1_000_000), sizes):
        assert 8 * n <= s <= (2 * (n // 4 + 1)) * 256 * 4 + 24 * n + (1 << 21)


def test_nothing_to_do_needs_no_arrays(sp):
    ok, lib = sp.SPMV_OK, sp._lib
    assert lib.spmv_q4_run(C.byref(q4(sp)), 0, 0, None, 64, None, 0, 0, None, 4, None) == ok
    empty = q4(sp, rows=0, codes=None, scales=None)
    assert lib.spmv_q4_run(C.byref(empty), 3, 0, None, 64, None, 0, 0, None, 0, None) == ok
    assert lib.spmv_q4_quantize(C.byref(empty), 0, None, 64, None, 0, None) == ok
    assert lib.spmv_embed(10, 16, 0, None, 16, 0, 4, None, 1.0, 0, None, 16, None) == ok
    assert lib.spmv_embed_grad(10, 16, 0, None, 16, 0, 4, None, 1.0, 1, 0, None, 16, None, 0,
                               None) == ok


def test_binding_refuses_host_tensors_and_wrong_types(sp):
    t = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        sp.spmv_embed(t, torch.zeros(2, dtype=torch.int64), torch.zeros(2, 32))
    with pytest.raises(ValueError):
        sp.spmv_q4_run(t, t, 32, t, t)
    with pytest.raises(ValueError):
        sp.spmv_q4_quantize(t, t, t, 32)
    with pytest.raises(ValueError):
        sp.spmv_embed_grad(t, torch.zeros(4, dtype=torch.int64), t)


class OnDevice:
    """What the binding looks at of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, rows, cols, dtype=torch.float32):
        self.shape, self.dtype = (rows, cols), dtype

    def stride(self):
        return self.shape[1], 1

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("codes,scales,zeros", [(64, 4, 4), (32, 4, 2), (64, 2, 2), (32, 2, 4),
                                                (31, 2, 2), (32, 1, 2), (33, 2, 2)])
def test_binding_refuses_a_matrix_of_another_width(sp, codes, scales, zeros):
    """Codes, scales or zero points of more or fewer columns than the vectors, the
    results or the dense matrix have (64)."""
    c, s = OnDevice(4, codes, torch.uint8), OnDevice(4, scales)
    z = OnDevice(4, zeros, torch.uint8)
    for call in (lambda: sp.spmv_q4_run(c, s, 32, OnDevice(1, 64), OnDevice(1, 4), zeros=z),
                 lambda: sp.spmv_q4_quantize(OnDevice(4, 64), c, s, 32, zeros=z),
                 lambda: sp.spmv_embed_q4(c, s, 32, None, OnDevice(4, 64), zeros=z)):
        with pytest.raises(ValueError):
            call()


def test_gradients_that_are_too_wide_are_refused_before_any_work(sp):
    """Before the sort's launch, so before the pointers are even looked up."""
    p, dim = 1 << 40, 64 * 65535 + 1
    call = lambda d: sp._lib.spmv_embed_grad(  # noqa: E731
        10, d, 0, p, d, 4, 4, 2 * p, 1.0, 0, 0, 3 * p, d, 4 * p, 1 << 35, None)
    assert call(dim) == sp.SPMV_ERR_TOO_LARGE
    assert call(dim - 1) != sp.SPMV_ERR_TOO_LARGE


# Arguments that are right but for their addresses, which are far apart and of no memory:
# without a GPU they reach the CUDA call that looks them up, so that what a test below makes
# wrong is what is refused. (With a GPU that call refuses the addresses.)
A = 1 << 32
GOOD = {
    "spmv_q4_run": lambda sp, m: [C.byref(m), 2, 0, 4 * A, 64, 5 * A, 4, 0, 6 * A, 4, None],
    "spmv_q4_quantize": lambda sp, m: [C.byref(m), 0, 4 * A, 64, 5 * A, 64, None],
    "spmv_embed_q4": lambda sp, m: [C.byref(m), 4, 4, 4 * A, 1.0, 0, 5 * A, 64, None],
    "spmv_embed": lambda sp, m: [10, 16, 0, 4 * A, 16, 4, 4, 5 * A, 1.0, 0, 6 * A, 16, None],
    "spmv_embed_grad": lambda sp, m: [10, 16, 0, 4 * A, 16, 4, 4, 5 * A, 1.0, 0, 0, 6 * A, 16,
                                      7 * A, 1 << 20, None],
}
MATRIX = dict(codes=A, scales=2 * A, zeros=3 * A, ld_zeros=2)


def answer(sp, name, at=None, value=None, **matrix):
    args = GOOD[name](sp, q4(sp, **{**MATRIX, **matrix}))
    if at is not None:
        args[at] = value
    return getattr(sp._lib, name)(*args)


def refused_for_this_alone(sp, name, *change, **matrix):
    if not torch.cuda.is_available():
        assert answer(sp, name) == sp.SPMV_ERR_CUDA
    assert answer(sp, name, *change, **matrix) == sp.SPMV_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["spmv_q4_run", "spmv_q4_quantize", "spmv_embed_q4"])
@pytest.mark.parametrize("bad", [{**b, "scales": 2 * A + 2} if "scales" in b and b["scales"]
                                 else b for b in BAD_Q4 if b.get("zeros") != 4096]
                         + [dict(ld_zeros=1)])
def test_one_fault_of_a_matrix_is_enough(sp, name, bad):
    refused_for_this_alone(sp, name, **bad)


@pytest.mark.parametrize("name,at,value", [
    ("spmv_q4_run", 1, -1), ("spmv_q4_run", 2, 3), ("spmv_q4_run", 3, None),
    ("spmv_q4_run", 3, 4 * A + 2), ("spmv_q4_run", 3, 6 * A - 4), ("spmv_q4_run", 4, 63),
    ("spmv_q4_run", 5, 6 * A + 4), ("spmv_q4_run", 5, 5 * A + 1), ("spmv_q4_run", 6, 3),
    ("spmv_q4_run", 7, -1), ("spmv_q4_run", 8, None), ("spmv_q4_run", 8, 6 * A + 2),
    ("spmv_q4_run", 8, A), ("spmv_q4_run", 8, 2 * A), ("spmv_q4_run", 8, 3 * A + 4),
    ("spmv_q4_run", 9, 3),
    ("spmv_q4_quantize", 1, 3), ("spmv_q4_quantize", 2, None), ("spmv_q4_quantize", 2, 4 * A + 1),
    ("spmv_q4_quantize", 2, A), ("spmv_q4_quantize", 2, 2 * A + 4), ("spmv_q4_quantize", 3, 63),
    ("spmv_q4_quantize", 4, 4 * A + 4), ("spmv_q4_quantize", 4, 3 * A + 4),
    ("spmv_q4_quantize", 5, 63),
    ("spmv_embed_q4", 1, -1), ("spmv_embed_q4", 2, 2), ("spmv_embed_q4", 3, 4 * A + 2),
    ("spmv_embed_q4", 5, 3), ("spmv_embed_q4", 6, None), ("spmv_embed_q4", 6, 5 * A + 1),
    ("spmv_embed_q4", 6, A), ("spmv_embed_q4", 6, 4 * A), ("spmv_embed_q4", 7, 63),
    ("spmv_embed", 0, -1), ("spmv_embed", 1, -1), ("spmv_embed", 2, 3), ("spmv_embed", 3, None),
    ("spmv_embed", 3, 4 * A + 2), ("spmv_embed", 4, 15), ("spmv_embed", 5, -1),
    ("spmv_embed", 6, 2), ("spmv_embed", 7, None), ("spmv_embed", 7, 5 * A + 2),
    ("spmv_embed", 9, -1), ("spmv_embed", 10, None), ("spmv_embed", 10, 4 * A + 4),
    ("spmv_embed", 10, 5 * A), ("spmv_embed", 11, 15),
    ("spmv_embed_grad", 0, -1), ("spmv_embed_grad", 1, -1), ("spmv_embed_grad", 2, 3),
    ("spmv_embed_grad", 3, None), ("spmv_embed_grad", 3, 4 * A + 2),
    ("spmv_embed_grad", 3, 6 * A + 4), ("spmv_embed_grad", 4, 15), ("spmv_embed_grad", 5, -1),
    ("spmv_embed_grad", 6, 16), ("spmv_embed_grad", 7, None), ("spmv_embed_grad", 7, 6 * A),
    ("spmv_embed_grad", 9, 2), ("spmv_embed_grad", 10, 3), ("spmv_embed_grad", 11, None),
    ("spmv_embed_grad", 12, 15), ("spmv_embed_grad", 13, None),
    ("spmv_embed_grad", 13, 7 * A + 8), ("spmv_embed_grad", 13, 4 * A),
    ("spmv_embed_grad", 14, 16)])
def test_one_fault_of_an_argument_is_enough(sp, name, at, value):
    refused_for_this_alone(sp, name, at, value)


def test_rows_without_tokens_are_no_more_than_the_table_has(sp):
    refused_for_this_alone(sp, "spmv_embed_q4", 3, None, rows=3)
    if not torch.cuda.is_available():
        assert answer(sp, "spmv_embed_q4", 3, None) == sp.SPMV_ERR_CUDA
