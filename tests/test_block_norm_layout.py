"""How the block norm's launches are laid out, over every dim that the entry
points accept: a program on the library's own planning functions (no GPU)."""
import os
import shutil
import subprocess

import pytest

from collective_communication_algorithms_gb300 import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "collective_communication_algorithms_gb300", "csrc")

# one line a shape: what it is for, then its layout
PROGRAM = r"""
#include <stdio.h>
#include "hc_ops.h"
using namespace hc;
static void show(const char* what, int dim, int es, const BlockNormRows& r) {
    const RowLayout& l = r.lay;
    printf("%s %d %d %d %d %d %d %d %d %d %d %d\n", what, dim, es, (int)r.access, r.cols, r.ops, l.tx, l.ty, l.cs,
           l.stages, l.slot, l.weights);
}
int main() {
    const long cases[][2] = {{40, 1}, {4096, 1}, {4096, 8}, {4096, 4096}, {200, 200}, {4096, 2048}};
    for (int dim = 1; dim <= (int)kBlockNormMaxDim; dim++)
        for (int es = 2; es <= 4; es += 2)
            for (int how = 0; how < 3; how++) {
                const bool vectors = how == 0, alike = how < 2;
                if (vectors && dim * es % 16) continue;
                show("forward", dim, es, block_norm_rows(dim, es, vectors, alike));
                for (const auto& c : cases)
                    for (int same = 0; same < 2; same++) {
                        BlockNormPlan q = block_norm_plan(c[0], dim, c[1], true, same);
                        show("gradient", dim, es, block_norm_grad_rows(&q, c[0], dim, es, vectors, alike));
                    }
            }
    return 0;
}
"""
ONE_BY_ONE, VECTORS, WINDOW = 0, 1, 2


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    cuda = "/usr/local/cuda/include"
    if shutil.which("g++") is None or not os.path.isdir(cuda):
        pytest.skip("g++ or the CUDA headers not found")
    from collective_communication_algorithms_gb300 import build
    build.build()
    d = tmp_path_factory.mktemp("layout")
    src, exe, lib = d / "layout.cpp", d / "layout", os.path.dirname(B.LIB_PATH)
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src),
                    "-L", lib, "-lhc", "-Wl,-rpath," + lib, "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    names = "dim es access cols ops tx ty cs stages slot weights".split()
    shapes = set(out.splitlines())
    return [dict(zip(names, map(int, line.split()[1:])), what=line.split()[0]) for line in sorted(shapes)]


def test_every_shape_can_be_launched(layouts):
    """Clusters of at most 8 blocks (what every GPU takes, and what the kernels
    keep room for), 512 threads and the shared memory of a block, and a thread
    for every column of the row with the columns that a window begins before
    it."""
    bad = []
    for s in layouts:
        wide = s["dim"] + (16 // s["es"] - 1 if s["access"] == WINDOW else 0)
        in_warp = 8 if s["what"] == "gradient" or s["stages"] else 16
        per_thread = s["cols"] if s["stages"] else in_warp
        shared = s["slot"] * s["ops"] * s["stages"] * s["ty"] + s["weights"]
        if not (s["cs"] <= 8 and s["tx"] * s["ty"] <= 512 and s["tx"] * s["cs"] * per_thread >= wide
                and shared <= 226 << 10 and (s["stages"] >= 1 or s["tx"] <= 32)):
            bad.append(s)
    assert not bad, "%d of %d, the first: %s" % (len(bad), len(layouts), bad[:3])


def test_rows_are_brought_ahead(layouts):
    """Every ring holds the row after the one under way."""
    bad = [s for s in layouts if s["stages"] == 1]
    assert not bad, "%d of %d, the first: %s" % (len(bad), len(layouts), bad[:3])
