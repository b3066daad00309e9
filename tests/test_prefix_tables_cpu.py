"""The bounds that the shared-prefix merge puts on its table entries, run on the host: an entry that no
CTA wrote holds whatever the scratch memory held."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "looped_transformer_self_b200", "csrc")

SOURCE = r"""
#include "attn_prefix.cuh"
#include <cstdio>
using namespace lt;
int main() {
  int rx, ry, rz, rw, head, group, max_tiles, mt, tx, ty, grid;
  while (scanf("%d %d %d %d %d %d %d %d %d %d %d", &rx, &ry, &rz, &rw, &head, &group, &max_tiles, &mt, &tx, &ty,
               &grid) == 11) {
    PrefixPlace p = {};
    if (!prefix_place(make_int4(rx, ry, rz, rw), head, group, max_tiles, mt, p)) puts("row");
    else if (!prefix_parts(make_int4(tx, ty, 0, 0), grid, p)) puts("tile");
    else printf("%d %d %d %d %d\n", p.t, p.r, p.first, p.parts, p.two);
  }
}
"""


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    from looped_transformer_self_b200 import build
    d = tmp_path_factory.mktemp("places")
    (d / "t.cu").write_text(SOURCE)
    subprocess.check_call([build.NVCC] + build.FLAGS + ["-I", CSRC, str(d / "t.cu"), "-o", str(d / "t")],
                          stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        return subprocess.run([str(d / "t")], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
    return run


BIG, F3 = 2**31 - 1, 0x40400000  # F3: the bits of 3.0f, what an earlier call's partials leave behind


def test_entries_as_written(places):
    #        row entry      head group max_tiles mt  tile entry grid
    cases = [((0, 1, 0, 1), 0, 1, 4, 16, (0, 3), 296), ((5, 2, 12, 1), 7, 4, 40, 64, (290, 6), 296),
             ((3, 1, 127, 2), 0, 1, 4, 256, (147, 1), 148), ((0, 1, 252, 1), 3, 4, 1, 256, (0, 148), 148)]
    got = places([r + (h, g, m, mt) + t + (grid,) for r, h, g, m, mt, t, grid in cases])
    assert got == ["0 0 0 3 1", "7 15 290 6 1", "3 127 147 2 2", "0 255 0 148 1"]


@pytest.mark.parametrize("row", [(-1, 0, 0, 1), (4, 0, 0, 1), (BIG, 1, 0, 1), (F3, F3, F3, F3), (0, BIG, 0, 1),
                                 (0, -BIG, 0, 1), (0, 1, -1, 1), (0, 1, 256, 1), (0, 1, BIG, 1), (0, 1, 128, 2),
                                 (2, 1, 0, 1), (-BIG - 1, -BIG - 1, -BIG - 1, 2)])
def test_stale_row_entries_are_refused(places, row):
    assert places([row + (9, 4, 4, 256, 0, 1, 148)]) == ["row"]  # head 9 of groups of 4: head 1 of key/value head 2


@pytest.mark.parametrize("tile", [(F3, F3), (BIG, 1), (BIG, BIG), (1, BIG), (0, 149), (148, 1), (147, 2), (-1, 1),
                                  (0, 0), (0, -1), (-BIG - 1, BIG), (100, -BIG - 1)])
def test_stale_tile_entries_are_refused(places, tile):
    assert places([(0, 1, 0, 1, 9, 4, 4, 256) + tile + (148,)]) == ["tile"]


def test_partials_stay_inside_the_scratch(places):
    """Whatever the entries, the last partial read lies in the grid + max_tiles slots of mt rows."""
    values = [-BIG - 1, -BIG, -5, -1, 0, 1, 2, 3, 7, 15, 16, 63, 127, 128, 129, 147, 148, 255, 256, F3, BIG - 1, BIG]
    cases = []
    for i, a in enumerate(values):
        for j, b in enumerate(values):
            c, d = values[(i * 7 + j * 3) % len(values)], values[(i + 5 * j) % len(values)]
            for head, group, mt in ((0, 1, 256), (9, 4, 256), (130, 64, 64), (5, 5, 16)):
                cases += [(a, b, c, 2, head, group, 7, mt, d % 160, 1 + j % 150, 148),
                          (i % 8, j % 3, c, d, head, group, 7, mt, a, b, 148)]
    for case, line in zip(cases, places(cases), strict=True):
        if line in ("row", "tile"):
            continue
        t, r, first, parts, two = map(int, line.split())
        mt, grid, max_tiles = case[7], case[10], case[6]
        last = (first + (parts - 1) // two + t) * mt + (parts - 1) % two * (mt // 2) + r
        assert 0 <= first and parts > 0 and 0 <= r and 0 <= t and last < (grid + max_tiles) * mt, case
