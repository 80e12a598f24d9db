"""kernel_choice's rules are the source's: each of its lines stands there as it was when
they were written."""
import os

import pytest

from nvfp4_block_scaled_route_amd import build as B

from . import kernel_choice as C

CSRC = os.path.join(B.PKG, "csrc")
LINES = {
    "fp8.hip": """
        if (T <= 16 && N <= 8192) return launch_fp8_skinny<1>(a, s);
        if (T <= 32 && N <= 4096) return launch_fp8_skinny<2>(a, s);
        const auto tiles = [&](int64_t rows, int64_t cols) { return (T + rows - 1) / rows * ((N + cols - 1) / cols); };
        if (tiles(64, 64) <= 256) return K > 2048 ? launch_fp8<2, 2, 1, 2>(a, s) : launch_fp8<2, 2, 2, 1>(a, s);
        if (tiles(64, 128) <= 256) return launch_fp8<2, 4, 1, 2>(a, s);
        if (tiles(64, 128) <= 512) return launch_fp8<2, 4, 1, 1>(a, s);
        if (tiles(128, 128) <= 512) return launch_fp8<4, 4, 1, 1>(a, s);
        return launch_fp8_wide(a, s);
    """,
    "grouped.hip": """
        const int held = (g.rows + bm - 1) / bm, all = (g.end - g.row + bm - 1 - bm / 2) / bm;
        g.tiles = g.end == g.row ? 0 : held > all ? held : all > 1 ? all : 1;
        if (gg_split(t, 320) < held && 15 * t.tiles * t.nt < 16 * g.tiles * g.nt) g = t;
        return blocks >= 1024 || 10 * blocks >= 8 * ((blocks + 255) / 256 * 256);
        const int64_t rows = rows_max / side + (rows_max < E ? rows_max : E) / 2, least = rows_max < E ? rows_max : E;
        return (rows > least ? rows : least) * ((cols + side - 1) / side);
        const int64_t wide = blocks(256);
        if (rows_max >= 32 * (int64_t)E && wide >= 200 && (wide >= 448 || (rows_max >= 96 * (int64_t)E && gg_filled(wide)))) return 256;
        if (rows_max >= 32 * (int64_t)E && blocks(128) >= 150) return 128;
        return 32;
        const int64_t wide = (int64_t)E * ((N + 255) / 256) * ((D + 255) / 256);
        if (rows_max >= (wide >= 4096 ? 96 : 192) * (int64_t)E && wide >= 200 && gg_filled(wide))
    """}


@pytest.mark.parametrize("name", LINES)
def test_rules_are_the_sources(name):
    with open(os.path.join(CSRC, name)) as f:
        source = " ".join(f.read().split())
    at = 0
    for line in filter(None, (" ".join(l.split()) for l in LINES[name].splitlines())):
        found = source.find(line, at)
        assert found >= 0, f"not there, or not in this order: {line}"
        at = found


def test_choices_at_known_sizes():
    assert C.fp8_gemm(1100, 3000, 528) == "64 x 128" and C.fp8_gemm(2048, 4096, 4096) == "128 x 128"
    assert C.fp8_gemm(4096, 4096, 4096) == "256 x 256" and C.fp8_gemm(517, 2085, 4112) == "64 x 128, two groups"
    assert C.grouped_side(3285, 8, 6400) == 128 and C.grouped_side(3285, 8, 7200) == 256
    assert C.grouped_side(48896, 128, 4096) == 256 and C.grouped_side(1024, 64, 1536) == 32
    assert C.grouped_tall(320, 320, 7200) and not C.grouped_tall(321, 321, 7200) and not C.grouped_tall(256, 256, 7200)
    assert C.weight_side(48896, 128, 4096, 1536) == 256 and C.weight_side(1000, 1, 136, 72) == 128
