"""The weight gradients' choice of a tile (on the CPU): among those that their
launcher has, the one of the least estimated time, with every group's row
tiles counted as they are."""
import math
import os
import random
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE = os.path.join(ROOT, "tiled_gemm_f32_amd", "csrc", "gemm_grouped_tile.hpp")
UNITS = 256


def part(text, start, end="\n}\n"):
    at = text.index(start)
    return text[at:text.index(end, at) + len(end)]


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    text = open(TILE).read()
    tmp = tmp_path_factory.mktemp("choice")
    (tmp / "t.cpp").write_text(
        "#include <algorithm>\n#include <cmath>\n#include <cstdio>\n" + part(text, "constexpr int kComputeUnits", ";\n") +
        part(text, "enum TileSize", ";\n") + part(text, "struct TileCost", "};\n") +
        part(text, "constexpr TileCost kTileCosts[]", "};\n") + part(text, "inline double tile_time") +
        part(text, "inline TileSize wgrad_tile") +
        "int main(){int n,k,g,large;double s,m;while(scanf(\"%d %d %d %lf %d %lf\",&n,&k,&g,&s,&large,&m)==6)"
        "{const TileCost &c=kTileCosts[wgrad_tile(n,k,g,s,large,m)];printf(\"%d %d\\n\",c.bm,c.bn);}}\n")
    exe = str(tmp / "t")
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", exe, str(tmp / "t.cpp")], check=True)

    def ask(calls):
        out = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in calls), capture_output=True, text=True,
                             check=True).stdout.split()
        return [(int(a), int(b)) for a, b in zip(out[::2], out[1::2])]
    return ask


def costs():
    table = part(open(TILE).read(), "constexpr TileCost kTileCosts[]", "};\n")
    return {(int(a), int(b)): (float(c), float(d), float(e)) for a, b, c, d, e in
            re.findall(r"\{(\d+), (\d+), ([\d.]+), ([\d.]+), ([\d.]+)\}", table)}


def launched():
    """Tiles that launch_wgrad launches: TileConfig<type, FM, FN, WM, WN, ...> is 32 FM WM x 32 FN WN."""
    body = part(open(TILE).read(), "hipError_t launch_wgrad")
    return {(32 * fm * wm, 32 * fn * wn) for fm, fn, wm, wn in
            (map(int, m) for m in re.findall(r"TileConfig<DT, (\d), (\d), (\d), (\d)", body))}


def test_only_tiles_that_are_launched_are_chosen_by_their_own_time(choice):
    have, cost = launched(), costs()
    assert have == {(256, 256), (128, 128), (64, 128)}
    rng = random.Random(2)
    calls = [(632, 2136, 3, 37, 1, 0.0), (248, 1944, 8, 15, 1, 0.0), (512, 1024, 4, 16, 1, 0.0)]
    for _ in range(3000):
        n, k = (int(2 ** rng.uniform(3, 13)) for _ in range(2))
        calls.append((n, k, rng.choice([1, 2, 3, 8, 40, 200]), rng.randrange(0, 300), rng.randrange(2),
                      rng.choice([0.0, 1.75])))
    for (n, k, groups, slabs, large, matrix), got in zip(calls, choice(calls)):
        def time(tile):
            slab, own, alone = cost[tile]
            turns = groups * math.ceil(n / tile[0]) * math.ceil(k / tile[1]) / UNITS
            turns = max(1.0, turns) if tile == (64, 128) else math.ceil(turns)
            least = matrix * tile[0] * tile[1] / 128 ** 2
            return max(turns * (slabs * max(slab, least) + 2 * own), slabs * max(alone, least) + 6)
        tiles = [t for t in have if large or t != (256, 256)]
        assert got in tiles and time(got) <= min(map(time, tiles)) * (1 + 1e-12), (n, k, groups, slabs, large, matrix)
    assert choice(calls[:3]) == [(128, 128), (128, 128), (64, 128)]
