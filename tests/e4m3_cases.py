"""Sizes that reach each kernel of the 8-bit product on 256 compute units, and
the planner (csrc/e4m3_plan.hpp) compiled for the host that says so."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Kernels by their names here: tiles in the planner's order, then the streaming
# kernels by the rows they hold.
TILES = ("256x256", "128x128", "64x128", "64x64")
SKINNY = ("rows16", "rows32", "rows64")
SLICE = {"256x256": 64, "128x128": 128, "64x128": 128, "64x64": 128}  # codes of K per stage
STAGES = {"256x256": 4, "128x128": 2, "64x128": 2, "64x64": 2}

# (kernel, M, N, K, rows 16-byte aligned, workspace, K splits).  K is at, below
# and past whole slices, a multiple of 16 and not, with fewer slices than stages
# and with more; M and N are ragged.
CASES = [
    ("256x256", 10639, 32304, 61, True, False, 1),
    ("256x256", 17027, 12418, 100, True, False, 1),
    ("256x256", 4619, 23836, 192, True, False, 1),
    ("256x256", 3301, 30007, 250, True, False, 1),
    ("256x256", 3300, 30000, 256, True, False, 1),
    ("256x256", 16390, 1703, 707, True, False, 1),
    ("256x256", 4001, 4003, 4000, True, False, 1),
    ("256x256", 12300, 129, 16400, True, True, 5),
    ("256x256", 12290, 131, 16391, True, True, 5),
    ("128x128", 27433, 2569, 61, True, False, 1),
    ("128x128", 16390, 1301, 200, True, False, 1),
    ("128x128", 4100, 4100, 1100, True, False, 1),
    ("128x128", 65, 16390, 1040, True, False, 1),
    ("128x128", 67, 521, 59999, True, True, 47),
    ("128x128", 30001, 2051, 61, False, False, 1),
    ("128x128", 3301, 6203, 200, False, False, 1),
    ("128x128", 65, 16390, 1037, False, False, 1),
    ("128x128", 67, 521, 59999, False, True, 47),
    ("64x128", 3301, 6203, 64, True, False, 1),
    ("64x128", 67, 8197, 250, True, False, 1),
    ("64x128", 65, 8200, 256, True, False, 1),
    ("64x128", 131, 8197, 1090, True, False, 1),
    ("64x128", 67, 131, 16390, True, True, 43),
    ("64x128", 3301, 6203, 61, False, False, 1),
    ("64x128", 67, 8197, 250, False, False, 1),
    ("64x128", 65, 8200, 300, False, False, 1),
    ("64x128", 67, 131, 16390, False, True, 43),
    ("64x64", 65, 65, 61, True, False, 1),
    ("64x64", 70, 200, 256, True, False, 1),
    ("64x64", 203, 515, 1037, True, False, 1),
    ("64x64", 67, 65, 2001, True, True, 16),
    ("64x64", 65, 65, 61, False, False, 1),
    ("64x64", 203, 515, 1037, False, False, 1),
    ("64x64", 67, 65, 2001, False, True, 16),
    ("rows16", 1, 300, 4096, True, True, 1),
    ("rows16", 16, 101, 1037, False, True, 1),
    ("rows32", 17, 515, 61, True, True, 1),
    ("rows32", 31, 101, 1037, False, True, 1),
    ("rows64", 33, 515, 130, True, True, 1),
    ("rows64", 63, 101, 301, False, True, 1),
]

_PROGRAM = r"""
#include <stdio.h>
#include "e4m3_plan.hpp"
using namespace sgemm;
int main(int argc, char **)
{
    if (argc == 1) {  // the kernels there are
        for (const E4m3Tile &t : kE4m3Tiles) printf("%dx%d %d\n", t.bm, t.bn, t.reg);
        for (const E4m3Skinny &s : kE4m3Skinny) printf("rows%d 1\n", s.rows);
        return 0;
    }
    int m, n, k, aligned, ws;
    while (scanf("%d %d %d %d %d", &m, &n, &k, &aligned, &ws) == 5) {
        // (a workspace is what the selector would like for aligned rows)
        const long long bytes = ws ? e4m3_plan(m, n, k, 256, true, LLONG_MAX).workspace_bytes : 0;
        const E4m3Plan p = e4m3_plan(m, n, k, 256, aligned, bytes);
        printf("%d %d %d\n", p.kernel, p.splits, p.k_chunk);
    }
}
"""


class Planner:
    """The planner, compiled with the host compiler into `folder`."""

    def __init__(self, folder):
        source, self.program = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan")
        with open(source, "w") as f:
            f.write(_PROGRAM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", f"-I{ROOT}/include",
                        f"-I{ROOT}/fp32_gemm_sgemm_amd/csrc", "-I/opt/rocm/include", source, "-o", self.program],
                       check=True)

    def kernels(self):
        """(name, whether it has a form for rows that are not aligned) of each."""
        out = subprocess.run([self.program], capture_output=True, text=True, check=True).stdout
        return [(name, reg == "1") for name, reg in (line.split() for line in out.splitlines())]

    def plans(self, sizes):
        """(kernel, splits, k_chunk) of each (M, N, K, aligned, workspace)."""
        text = "\n".join(" ".join(str(int(v)) for v in s) for s in sizes)
        out = subprocess.run([self.program, "-"], input=text, capture_output=True, text=True, check=True).stdout
        plans = [tuple(int(v) for v in line.split()) for line in out.splitlines()]
        return [(TILES[k] if k >= 0 else SKINNY[-1 - k], s, c) for k, s, c in plans]
