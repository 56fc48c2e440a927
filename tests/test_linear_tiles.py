"""The rule that picks gdn_linear_act's tile, compiled on the host: the sizes of the GPU test reach every tile shape, gated and
not, with K in one part and in several."""

import os
import shutil
import subprocess

import pytest

from tests.test_gpu_linear_tiles import SIZES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_verify_amd", "csrc")
MAIN = """
#include <cstdio>
#include "gdn_tiles.h"
int main()
{
    long long M, N, K;
    int elem, gated;
    while (scanf("%lld %lld %lld %d %d", &M, &N, &K, &elem, &gated) == 5) {
        const gdn::Choice c = gdn::choose_tile(M, N, K, elem, gated != 0);
        printf("%d %d\\n", c.tile, c.splits);
    }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    at = tmp_path_factory.mktemp("tiles")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + CSRC, str(at / "main.cpp"), "-o", str(at / "main")], check=True)

    def of(sizes):
        text = "".join(f"{M} {N} {K} {2 if t == 'bf16' else 1} {int(g)}\n" for M, N, K, t, g in sizes)
        r = subprocess.run([str(at / "main")], input=text, capture_output=True, text=True, check=True, timeout=60)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    return of


# in the order of gdn::Tile: rows of a tile, columns (w's rows), and whether K is cut into parts somewhere for it
TILES = [(16, 64, True), (16, 64, False), (32, 64, True), (64, 64, True), (64, 128, True), (128, 128, True), (128, 128, True), (256, 256, True)]


def test_every_tile_is_reached(choose):
    got = choose(SIZES)
    assert len(got) == len(SIZES)
    for tile, (bm, _, parts) in enumerate(TILES):
        mine = [(s, c[1]) for s, c in zip(SIZES, got) if c[0] == tile]
        assert {g for (_, _, _, _, g), _ in mine} == {False, True}, tile
        assert {t for (_, _, _, t, _), _ in mine} == {"bf16", "e4m3", "i8"}, tile
        assert any(sp > 1 for _, sp in mine) == parts and any(sp == 1 for _, sp in mine), tile
        assert any(N % 4 for (_, N, _, _, _), _ in mine) and any(N % 4 == 0 for (_, N, _, _, _), _ in mine), tile
        assert all(K * (2 if t == "bf16" else 1) % 128 for (_, _, K, t, _), _ in mine), tile  # K ends inside a step
        if bm > 32:
            assert any(M % bm == 1 for (M, _, _, _, _), _ in mine), tile
        if bm >= 64:
            assert any(M > 8 * bm for (M, _, _, _, _), _ in mine), tile
    assert any(M % bm == bm - 1 for (M, _, _, _, _), c in zip(SIZES, got) for bm in (TILES[c[0]][0],) if bm == 256)


def test_parts_of_k_are_whole_steps(choose):
    """Every part has at least one step, and there are no more parts than a launch's y axis holds."""
    sizes = [(m, n, k, t, g) for m in (1, 16, 17, 33, 64, 65, 300, 1024, 8191) for n in (1, 60, 1000, 5120, 40_000)
             for k in (16, 144, 4096, 131_056, (1 << 26) - 16) for t in ("bf16", "e4m3") for g in (False, True)]
    for (_, _, k, t, _), (tile, splits) in zip(sizes, choose(sizes)):
        steps = -(-k * (2 if t == "bf16" else 1) // 128)
        assert 0 <= tile < len(TILES) and 1 <= splits <= min(steps, 480)
