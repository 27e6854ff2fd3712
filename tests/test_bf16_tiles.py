"""Which kernel a bf16 expert product takes: the rule, compiled for the host, on the cases that the GPU tests
hold each kernel to, so that a change of the rule cannot leave a kernel without them."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from block_scaled_fp4_02_amd import build
from tests import bf16_cases as cases

PROGRAM = r"""
#include <stdio.h>
#include "bf16_tiles.hpp"
int main() {
  int what, E, N, K, epilogue, transposed;
  long long R;
  while (scanf("%d %d %d %d %lld %d %d", &what, &E, &N, &K, &R, &epilogue, &transposed) == 7)
    printf("%d\n", what ? static_cast<int>(moe::bf16::wgrad_large(E, N, K, R))
                        : static_cast<int>(moe::bf16::gemm_tile(E, N, R, static_cast<moe::bf16::Epilogue>(epilogue), transposed)));
}
"""
EPILOGUES = {cases.PLAIN: 0, cases.GATED: 1, cases.BACK: 2}   # in the order of Epilogue


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("tiles")
    (at / "tiles.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, str(at / "tiles.cpp"), "-o", str(at / "tiles")], check=True)

    def run(questions):
        text = "\n".join(" ".join(map(str, q)) for q in questions)
        return [int(v) for v in subprocess.run([str(at / "tiles")], input=text, capture_output=True, text=True, check=True).stdout.split()]
    return run


def test_every_kernel_has_its_cases(ask):
    questions = []
    for way, tile, K in cases.CASES:
        sizes, N = cases.sizes_of(way, tile)
        epilogue, layout = cases.WAYS[way]
        questions.append((0, len(sizes), N, K, sum(sizes) + cases.PAD, EPILOGUES[epilogue], int(layout == cases.TRANSPOSED)))
    assert [cases.TILES[t] for t in ask(questions)] == [tile for _, tile, _ in cases.CASES]


def test_the_rule_names_no_other_kernel(ask):
    """Over a grid of sizes: each epilogue and layout stays among the kernels that it has, and reaches them all."""
    for way, (epilogue, layout) in cases.WAYS.items():
        grid = [(0, E, N, 64, R, EPILOGUES[epilogue], int(layout == cases.TRANSPOSED))
                for E in (1, 2, 7, 32, 256, 1024) for N in (16, 128, 784, 2048, 6144, 1 << 20) for R in (1, 3, 16, 40, 128, 300, 1024, 9000, 100000, 1 << 30)]
        assert {cases.TILES[t] for t in ask(grid)} == set(cases.taken(way)), way


def test_no_rows(ask):
    assert all(0 <= t < len(cases.TILES) for t in ask([(0, 4, 128, 64, 0, e, t) for e in range(3) for t in (0, 1)]))
    assert ask([(1, 4, 4096, 4096, 0, 0, 0)]) == [0]
