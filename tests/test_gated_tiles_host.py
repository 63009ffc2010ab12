"""Which kernel takes a gated product, by the rule in csrc/gated_tiles.hpp compiled on the host (CPU only): every shape of
the GPU tests of a tile's form has that tile on a card of 256 CUs, six stages at least and more tiles than CUs."""
import os
import subprocess

import pytest

from fp8_dynamic_scaling_amd import build as hb
from tests import test_gpu_gated_tiles as shapes

PROGRAM = """
#include <cstdio>
#include "gated_tiles.hpp"
int main() {
  long M, F, K;
  int E, packed, exact;
  while (std::scanf("%ld %ld %ld %d %d %d", &M, &F, &K, &E, &packed, &exact) == 6)
    std::printf("%d\\n", fp8dyn::gated_tile_rows(M, F, K, E, packed, exact, 256));
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(hb.HERE, "csrc"), "-o", str(d / "rule"), str(d / "rule.cpp")],
                   check=True)

    def rows(*queries):
        text = "\n".join(" ".join(str(int(x)) for x in q) for q in queries)
        r = subprocess.run([str(d / "rule")], input=text, capture_output=True, text=True, check=True)
        return [int(x) for x in r.stdout.split()]

    return rows


def test_dense_shapes(rule):
    for tile, M, F, K, packed in shapes.DENSE:
        assert rule((M, F, K, 0, packed, 0), (M, F, K, 0, packed, 1)) == [tile, tile], (tile, M, F, K)
        assert K > 5 * 64 and -(-M // tile) * -(-F // 128) > 256


def test_grouped_shapes(rule):
    for tile, rows, pad, F, K, packed in shapes.GROUPED:
        M, E = sum(rows) + pad, len(rows)
        assert rule((M, F, K, E, packed, 0), (M, F, K, E, packed, 1)) == [tile, tile], (tile, rows, F, K)
        assert K > 5 * 64 and sum(-(-r // tile) for r in rows) * -(-F // 128) > 256


def test_every_form_is_listed():
    for tile in (64, 128, 256):
        for packed in (True, False):
            assert any(c[0] == tile and c[-1] == packed for c in shapes.DENSE)
            assert any(c[0] == tile and c[-1] == packed for c in shapes.GROUPED)
        assert {c[3] % 64 for c in shapes.DENSE if c[0] == tile and not c[4]} == {16, 32, 48}


def test_ends_of_the_rule(rule):
    """Few rows, short sums and weights past 32-bit offsets."""
    assert rule((1, 14336, 4096, 0, 1, 0), (32, 14336, 4096, 0, 0, 1), (300, 66000, 16400, 0, 0, 0)) == [0, 0, 0]
    assert rule((1000, 512, 64, 3, 0, 0), (300, 66000, 16400, 3, 0, 1)) == [-1, -1]
    assert rule((8192, 14336, 4096, 0, 1, 0), (32768, 7168, 2048, 32, 1, 0)) == [256, 256]
