"""The example that runs the dense-table operators together: training lowers the
loss well below that of guessing, the 4-bit model keeps it, and what it decodes
follows the chain it was trained on."""
import importlib.util
import math
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


def test_bigram_example():
    from conftest import build_library
    build_library()
    spec = importlib.util.spec_from_file_location(
        "bigram_q4", os.path.join(ROOT, "examples", "bigram_q4.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    r = mod.main(["--vocab", "500", "--dim", "128", "--steps", "150", "--batch", "4096"])
    assert abs(r["first"] - math.log(500)) < 0.5  # the start guesses
    assert r["last"] < 0.6 * r["first"] and r["dense"] < 0.6 * r["first"]
    assert r["quant"] < r["dense"] + 0.2
    assert r["likely"] >= 0.9 * r["decoded"]
