"""Host-side rules of the serving operators' launches (no GPU needed): a small C++ program
over csrc/serving.h prints what they choose."""
import os
import subprocess

import pytest

from pack_mla_cache_gb300 import build as B

MAIN = r"""
#include "serving.h"
#include <cstdio>
#include <cstdlib>
int main(int, char** v) {
  std::printf("%d\n", mla::attention_tile_rows(std::atoi(v[1]), std::atoi(v[2]), std::atoi(v[3]),
                                               std::atoi(v[4]) != 0));
}
"""


@pytest.fixture(scope="module")
def tile_rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("serving_host")
    (d / "main.cpp").write_text(MAIN)
    include = os.path.join(os.path.dirname(B.cuda_lib_dir()), "include")
    subprocess.run(["g++", "-std=c++17", "-O0", "-I", B.CSRC, "-I", B.INCLUDE, "-I", include,
                    str(d / "main.cpp"), "-o", str(d / "main")], check=True)
    return lambda *a: int(subprocess.run([str(d / "main"), *map(str, a)], check=True,
                                         capture_output=True, text=True).stdout)


@pytest.mark.parametrize("tokens,heads,seqs,fp8,want", [
    (1, 16, 1, 0, 16), (64, 16, 64, 0, 16), (65, 16, 64, 0, 32), (1, 128, 1, 0, 64),
    (1, 128, 1, 1, 32), (2048, 16, 2, 0, 64), (4, 8, 1, 0, 32),
    (2 ** 31 - 1, 1, 1, 0, 64), (2 ** 31 - 1, 1, 4096, 0, 64), (2 ** 31 - 1, 1, 4096, 1, 32),
])
def test_rows_of_a_query_tile(tile_rows, tokens, heads, seqs, fp8, want):
    assert tile_rows(tokens, heads, seqs, fp8) == want
