"""Which kernel an 8-bit product takes, without a GPU: the rule, cut out of its source and compiled for
the host, chooses for each size that the GPU tests name the kernel that they name it for, and those
are all there are."""
import os
import shutil
import subprocess

import pytest

pytest.importorskip("torch")
B = pytest.importorskip("bit_weight_only_w4a16_amd.build")
pytest.importorskip("bit_weight_only_w4a16_amd.int8")

from test_gpu_ffn_edges import ROWS, TILES  # noqa: E402

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")

MAIN = r"""
int main() {
  for (const Tile& t : kTiles) printf("%dx%d %d\n", t.bm, t.bn, t.teams);
  printf("--\n");
  long m, n, k;
  while (scanf("%ld %ld %ld", &m, &n, &k) == 3) {
    const Choice c = choose(m, n, k);
    if (c.tile < 0) printf("rows\n");
    else printf("%dx%d %d %d\n", kTiles[c.tile].bm, kTiles[c.tile].bn, kTiles[c.tile].teams, c.splits);
  }
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """(the tiles there are, what the rule chooses for TILES and then ROWS in their order)"""
    text = open(os.path.join(B.CSRC, "gemm_i8.hip")).read()
    begin, end = text.index("struct Tile {"), text.index("hipError_t launch_tiles(")
    body = text[begin:text.rindex("template <", begin, end)]
    where = tmp_path_factory.mktemp("choice")
    source, exe = where / "choice.cpp", where / "choice"
    source.write_text("#include <math.h>\n#include <stdint.h>\n#include <stdio.h>\n#include <initializer_list>\n"
                      "constexpr int kI8Unit = 64;\nconst char* tuning_env(const char*) { return nullptr; }\n" + body + MAIN)
    subprocess.run(["g++", "-O2", "-std=c++17", str(source), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], input="\n".join("%d %d %d" % s for s in [*TILES.values(), *ROWS]), capture_output=True,
                         text=True, check=True).stdout
    kinds, chosen = out.split("--\n")
    return kinds.splitlines(), chosen.splitlines()


def test_sizes_choose_what_they_are_named_for(rule):
    for ((tile, teams, split), size), got in zip(TILES.items(), rule[1]):
        assert got.rsplit(" ", 1)[0] == f"{tile} {teams}" and (int(got.rsplit(" ", 1)[1]) > 1) == split, (size, got)


def test_every_tile_is_named(rule):
    assert {f"{tile} {teams}" for tile, teams, _ in TILES} == set(rule[0])
    assert len(TILES) == 2 * len(rule[0])   # each whole and split


def test_sizes_are_ragged_and_longer_than_a_turn_of_the_loop(rule):
    for ((tile, teams, _), (m, n, k)), got in zip(TILES.items(), rule[1]):
        steps = -(-k // 64) // (teams * int(got.split()[-1]))
        assert steps > 12 and m % 32 and n % 64 and k % 64, (tile, m, n, k)


def test_few_rows_take_the_kernel_for_them(rule):
    assert rule[1][len(TILES):] == ["rows"] * len(ROWS)
