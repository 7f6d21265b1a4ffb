"""How the launches of 4-bit products are split (host code of the library, asked with
what a GB300 holds: no GPU needed): the products whose tests mean the multi-phase form
take it, and every plan fits the shared memory."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT, build_library
from test_gpu_q4 import PHASED

PROGRAM = r"""
#include <cstdio>
#include "q4.h"
using namespace spmv::q4;
template <int NT>
Plan plan(const RunArgs& p, int columns, bool aligned, const Residency& r) {
  const int pitch = kStepColsOf<NT> / 2 + (aligned ? 0 : 16);
  return make_plan(p, columns, kStepColsOf<NT>, kWarps * kStagesOf<NT> * kTileRows * pitch, r);
}
int main() {
  Residency r;  // clusters of 1, 2, 4, 8 blocks at a time, one or two to an SM, as one GB300 said
  const int clusters[4][2] = {{152, 304}, {76, 152}, {36, 74}, {15, 36}};
  for (int i = 0; i < 8; ++i) r.clusters[i / 2][i % 2] = clusters[i / 2][i % 2];
  int rows, cols, n, parts, aligned;
  while (std::scanf("%d %d %d %d %d", &rows, &cols, &n, &parts, &aligned) == 5) {
    RunArgs p{};
    p.a.rows = rows;
    p.a.cols = cols;
    p.n = n;
    const Plan q = n * parts <= 8 ? plan<1>(p, n * parts, aligned != 0, r)
                                  : plan<2>(p, n * parts, aligned != 0, r);
    std::printf("%d %d %d %lld %lld %d %zu\n", q.P, q.steps, q.phaseSteps, q.tiles, q.clusters,
                q.maxTiles, q.smem);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans([(rows, cols, n, parts, aligned)]) -> [dict]"""
    lib = build_library()
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cu").write_text(PROGRAM)
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.run([nvcc, "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "spmv_sparse_storage_gb300", "csrc"), "-o",
                    str(at / "plan"), str(at / "plan.cu"), lib, "-Xlinker",
                    "-rpath=" + os.path.dirname(lib)], check=True, capture_output=True)

    def ask(shapes):
        lines = "".join(" ".join(str(int(v)) for v in s) + "\n" for s in shapes)
        out = subprocess.run([str(at / "plan")], input=lines, capture_output=True, text=True,
                             check=True).stdout.splitlines()
        names = ("P", "steps", "phase_steps", "tiles", "clusters", "max_tiles", "smem")
        return [dict(zip(names, map(int, line.split()))) for line in out]

    return ask


def test_products_meant_for_several_phases_have_them(plans):
    asked = [(rows, cols, n, 3 if x_type == "f32" else 1, ((cols + 1) // 2 + pad) % 16 == 0)
             for rows, cols, n, x_type, _, _, pad, _, _ in PHASED]
    assert {bool(a[4]) for a in asked} == {True, False}
    for (case, q) in zip(PHASED, plans(asked)):
        assert q["P"] == case[-1], case
        assert q["phase_steps"] < q["steps"] // q["P"], case


def test_plans_fit(plans):
    """Of any shape: a plan is found, it covers the matrix and stays within what a block
    may have (227 KB)."""
    sizes = (1, 31, 33, 1000, 5003, 70_001, 2 ** 31 - 1)
    asked = [(rows, cols, n, parts, aligned) for rows in sizes for cols in (0,) + sizes
             for n, parts in ((1, 1), (8, 1), (9, 1), (16, 1), (1, 3), (2, 3), (3, 3), (5, 3))
             for aligned in (0, 1)]
    for case, q in zip(asked, plans(asked)):
        assert q["P"] in (1, 2, 4, 8) and q["P"] <= max(q["steps"], 1), case
        assert q["phase_steps"] >= 1 and 0 < q["smem"] <= 227 * 1024, case
        assert q["clusters"] >= 1 and q["clusters"] * q["max_tiles"] >= q["tiles"], case
        assert q["clusters"] * q["P"] < 2 ** 31, case
