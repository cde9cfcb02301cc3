"""Sizes that reach each kernel of the gated 8-bit block on 256 compute units:
(kernel, M, N, K, rows 16-byte aligned, workspace, K splits), as in e4m3_cases,
N columns of each weight; and the block's planner, compiled for the host."""
import os
import subprocess

import e4m3_cases

E4M3_GATED = [
    ("256x256", 3506, 11106, 256, True, False, 1),
    ("256x256", 19727, 2409, 250, True, False, 1),
    ("256x256", 10639, 16152, 61, True, False, 1),
    ("256x256", 454, 12455, 2001, True, False, 1),
    ("256x256", 16408, 98, 9000, True, True, 3),
    ("256x256", 12808, 69, 16390, True, True, 5),
    ("128x128", 19873, 1796, 61, True, False, 1),
    ("128x128", 463, 14377, 250, True, False, 1),
    ("128x128", 205, 12341, 500, True, False, 1),
    ("128x128", 16497, 35, 1037, True, False, 1),
    ("128x128", 65, 8760, 4000, True, True, 3),
    ("128x128", 2090, 34, 16390, True, True, 15),
    ("128x128", 14491, 2188, 61, False, False, 1),
    ("128x128", 205, 12341, 500, False, False, 1),
    ("128x128", 16898, 33, 1040, False, False, 1),
    ("128x128", 65, 8760, 4000, False, True, 3),
    ("64x128", 660, 15909, 61, True, False, 1),
    ("64x128", 66, 12444, 200, True, False, 1),
    ("64x128", 8663, 33, 256, True, False, 1),
    ("64x128", 8500, 33, 1037, True, False, 1),
    ("64x128", 65, 3096, 2001, True, True, 4),
    ("64x128", 17, 548, 16390, True, True, 43),
    ("64x128", 580, 14166, 61, False, False, 1),
    ("64x128", 66, 12444, 200, False, False, 1),
    ("64x128", 8341, 34, 500, False, False, 1),
    ("64x128", 530, 35, 9000, False, True, 24),
    ("64x64", 65, 33, 61, True, False, 1),
    ("64x64", 70, 100, 256, True, False, 1),
    ("64x64", 203, 258, 1037, True, False, 1),
    ("64x64", 65, 1, 2001, True, True, 16),
    ("64x64", 65, 33, 61, False, False, 1),
    ("64x64", 203, 258, 1037, False, False, 1),
    ("64x64", 17, 1, 4000, False, True, 32),
    ("rows16", 1, 300, 4096, True, True, 1),
    ("rows16", 16, 101, 1037, False, True, 1),
    # (from 4081 columns on a workgroup takes 16 of each weight instead of 8)
    ("rows16", 9, 4080, 1037, False, True, 1),
    ("rows16", 2, 4081, 600, True, True, 1),
    ("rows16", 5, 8195, 1037, False, True, 1),
    ("rows16", 16, 9, 300, True, True, 1),
    ("rows16", 3, 7, 61, False, True, 1),
    ("rows32", 17, 515, 1050, True, False, 1),
    ("rows32", 31, 101, 1037, False, False, 1),
    ("rows64", 33, 515, 2002, True, False, 1),
    ("rows64", 63, 101, 4001, False, False, 1),
]


class Planner(e4m3_cases.Planner):
    """e4m3_cases' planner for the gated block's plans."""

    def __init__(self, folder):
        source, self.program = os.path.join(folder, "gated.cpp"), os.path.join(folder, "gated")
        with open(source, "w") as f:
            f.write(e4m3_cases._PROGRAM.replace("e4m3_plan(", "e4m3_gated_plan("))
        root = e4m3_cases.ROOT
        subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", f"-I{root}/include",
                        f"-I{root}/fp32_gemm_sgemm_amd/csrc", "-I/opt/rocm/include", source, "-o", self.program],
                       check=True)
